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
#include <algorithm>
#include <cooperative_groups.h>
#include <cstdint>
#include <type_traits>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "mx.h"
#include "mx_device.cuh"
#include "mx_internal.h"

namespace mxnorm {

using namespace mxk;
namespace cg = cooperative_groups;

struct NormParams {
    const void *x, *res;
    int64_t rows, ldx, ldr, ldh, ldy;
    uint32_t cols, vecs;       // vecs = cols / 8
    const void *w;
    int w_f32;
    float eps, inv_cols;
    void *h, *y;
    float *rstd;
    uint8_t *codes, *scales;
    int fmt, sl;
    uint32_t key;              // stochastic-rounding seed key
    uint32_t k_blocks, k_groups;
    bool word_scales;          // scale words are aligned
    bool wide;                 // fp32: every row starts on a 32-byte boundary
    uint64_t codes_cap, scales_cap;
};

// The kernels of this unit may be launched while the stream's last kernel still
// runs (programmatic serialization, which saves 1 to 3 us between short ones);
// they touch no global memory before it has ended and its writes are visible,
// and let their own successor be launched in the same way.
__device__ __forceinline__ void after_predecessor() {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

// Two fp32 values in a register pair, and IEEE operations on both at a time.
using f2 = uint64_t;
__device__ __forceinline__ f2 pair(float lo, float hi) {
    f2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
    return r;
}
__device__ __forceinline__ void unpair(f2 v, float &lo, float &hi) { asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v)); }
__device__ __forceinline__ f2 add2(f2 a, f2 b) {
    f2 r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ f2 mul2(f2 a, f2 b) {
    f2 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ f2 fma2(f2 a, f2 b, f2 c) {
    f2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {     // nearest even
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

// Eight consecutive values as loaded: four words of bf16 or eight of fp32.
template <bool BF16> struct Raw {
    uint4 v[BF16 ? 1 : 2];

    // wide: fp32 values on a 32-byte boundary, as one access (two halves would
    // each touch every 32-byte sector of the warp's)
    __device__ __forceinline__ void load(const void *base, int64_t off, bool wide) {
        if (!BF16 && wide) {
            asm volatile("ld.global.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                         : "=r"(v[0].x), "=r"(v[0].y), "=r"(v[0].z), "=r"(v[0].w), "=r"(v[!BF16].x), "=r"(v[!BF16].y),
                           "=r"(v[!BF16].z), "=r"(v[!BF16].w)
                         : "l"(static_cast<const float *>(base) + off)
                         : "memory");
            return;
        }
#pragma unroll
        for (int i = 0; i < (BF16 ? 1 : 2); ++i)
            v[i] = BF16 ? *reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(base) + off)
                        : reinterpret_cast<const uint4 *>(static_cast<const float *>(base) + off)[i];
    }
    __device__ __forceinline__ void zero() {
#pragma unroll
        for (int i = 0; i < (BF16 ? 1 : 2); ++i) v[i] = make_uint4(0u, 0u, 0u, 0u);
    }
    __device__ __forceinline__ void store(void *base, int64_t off, bool wide) const {
        if (!BF16 && wide) {
            asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(static_cast<float *>(base) + off),
                         "r"(v[0].x), "r"(v[0].y), "r"(v[0].z), "r"(v[0].w), "r"(v[!BF16].x), "r"(v[!BF16].y), "r"(v[!BF16].z),
                         "r"(v[!BF16].w)
                         : "memory");
            return;
        }
#pragma unroll
        for (int i = 0; i < (BF16 ? 1 : 2); ++i)
            if (BF16) *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(base) + off) = v[i];
            else reinterpret_cast<uint4 *>(static_cast<float *>(base) + off)[i] = v[i];
    }
    __device__ __forceinline__ void widen(f2 (&f)[4]) const {
        if (BF16) {
            const uint32_t w[4] = {v[0].x, v[0].y, v[0].z, v[0].w};
#pragma unroll
            for (int i = 0; i < 4; ++i) f[i] = pair(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
        } else {
            const uint32_t w[8] = {v[0].x, v[0].y, v[0].z, v[0].w, v[!BF16].x, v[!BF16].y, v[!BF16].z, v[!BF16].w};
#pragma unroll
            for (int i = 0; i < 4; ++i) f[i] = pair(__uint_as_float(w[2 * i]), __uint_as_float(w[2 * i + 1]));
        }
    }
    // rounded to the type
    __device__ __forceinline__ void narrow(const f2 (&f)[4]) {
        float a[8];
#pragma unroll
        for (int i = 0; i < 4; ++i) unpair(f[i], a[2 * i], a[2 * i + 1]);
        if (BF16) {
            v[0] = make_uint4(pack_bf16(a[0], a[1]), pack_bf16(a[2], a[3]), pack_bf16(a[4], a[5]), pack_bf16(a[6], a[7]));
        } else {
            v[0] = make_uint4(__float_as_uint(a[0]), __float_as_uint(a[1]), __float_as_uint(a[2]), __float_as_uint(a[3]));
            v[!BF16] = make_uint4(__float_as_uint(a[4]), __float_as_uint(a[5]), __float_as_uint(a[6]), __float_as_uint(a[7]));
        }
    }
    // this + b, rounded to the type (for bf16 the same as an fp32 sum rounded to
    // bf16: where the fp32 sum of two bf16 values is not exact, the smaller one
    // is below 2^-15 of the larger and cannot decide the rounding)
    __device__ __forceinline__ void add(const Raw &b) {
        if (BF16) {
            uint32_t *w = reinterpret_cast<uint32_t *>(v);
            const uint32_t *o = reinterpret_cast<const uint32_t *>(b.v);
#pragma unroll
            for (int i = 0; i < 4; ++i) asm("add.rn.bf16x2 %0, %0, %1;" : "+r"(w[i]) : "r"(o[i]));
        } else {
            f2 x[4], y[4];
            widen(x);
            b.widen(y);
#pragma unroll
            for (int i = 0; i < 4; ++i) x[i] = add2(x[i], y[i]);
            narrow(x);
        }
    }
};

// Eight weights, widened: the type is the weight's own.
__device__ __forceinline__ void load_weight8(const void *w, int w_f32, uint32_t col, f2 (&f)[4]) {
    if (w_f32) {
        Raw<false> r;
        r.load(w, col, false);
        r.widen(f);
    } else {
        Raw<true> r;
        r.load(w, col, false);
        r.widen(f);
    }
}

// Sum over the CTA, in an order fixed by its shape; every thread gets it.  All
// warps read the warps' sums as they are broadcast, which takes less time than
// a second round of shuffles.  `red` holds 32 floats that no other sum in
// flight uses, zero where there is no warp.
__device__ __forceinline__ float cta_sum(float s, float *red) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    const int nw = blockDim.x >> 5;
    if (nw == 1) return s;
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = s;
    __syncthreads();
    float4 t = *reinterpret_cast<const float4 *>(red);
    for (int i = 4; i < nw; i += 4) {
        const float4 u = *reinterpret_cast<const float4 *>(red + i);
        t.x += u.x;
        t.y += u.y;
        t.z += u.z;
        t.w += u.w;
    }
    return (t.x + t.y) + (t.z + t.w);
}
// Clears the places of the sums; the caller has a barrier before the first.
__device__ __forceinline__ void clear_sums(float (&red)[2][32]) {
    for (int i = threadIdx.x; i < 64; i += blockDim.x) red[i >> 5][i & 31] = 0.0f;
    __syncthreads();
}

// Codes of eight values to byte `off` of the codes; s is their block's scale code
// (the exponent + 127) when the block holds no NaN or Inf.
template <int FMT, bool SR>
__device__ __forceinline__ void encode8(const NormParams &p, uint64_t off, uint64_t index, const f2 (&y)[4], uint32_t s,
                                        bool store, bool nan_block) {
    constexpr int BITS = Fmt<FMT>::bits;
    constexpr int SLOT = BITS == 4 ? 4 : 8;
    float u[8];
    const float down = __uint_as_float((254u - s) << 23);      // 2^-e: s <= 254 - emax, and INT8 takes the other way
    const f2 f = pair(down, down);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        f2 r = y[i];
        if (Fmt<FMT>::emax != 0) asm("mul.rn.ftz.f32x2 %0, %1, %2;" : "=l"(r) : "l"(y[i]), "l"(f));
        unpair(r, u[2 * i], u[2 * i + 1]);
    }
    if (Fmt<FMT>::emax == 0) {
#pragma unroll
        for (int i = 0; i < 8; ++i) u[i] = scale_down<FMT>(u[i], static_cast<int>(s) - 127);
    }
    uint32_t pw[2];
    if (SR) {
        const uint32_t g = static_cast<uint32_t>(index >> 2);
#pragma unroll
        for (int j = 0; j < 2; ++j)
            pw[j] = sr_quad<FMT>(u[4 * j], u[4 * j + 1], u[4 * j + 2], u[4 * j + 3], fmix32((g + j) ^ p.key));
    } else {
#pragma unroll
        for (int j = 0; j < 2; ++j)
            pw[j] = cvt_pair<FMT>(u[4 * j], u[4 * j + 1]) | (cvt_pair<FMT>(u[4 * j + 2], u[4 * j + 3]) << (2 * SLOT));
    }
    if (nan_block) pw[0] = pw[1] = 0u;
    if (!store || !in_bounds(off, BITS, p.codes_cap)) return;
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

// The cast of eight values of vector `vec`, four of which are a 32-block in
// neighbouring lanes: they share the largest magnitude (as bits: non-negative
// floats order as integers, and an Inf or NaN is at or above 0x7f800000), and
// a group of four blocks its scale word, which is one word in every layout.
// row_at: the row's part of the scale's offset.  All lanes of the warp call this.
template <int FMT, bool SR>
__device__ __forceinline__ void cast8(const NormParams &p, int64_t row, uint32_t row_at, uint32_t vec, const f2 (&y)[4]) {
    float m = 0.0f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        float lo, hi;
        unpair(y[i], lo, hi);
        m = max_abs3(m, lo, hi);
    }
    uint32_t a = __float_as_uint(m);
    a = max(a, __shfl_xor_sync(0xffffffffu, a, 1));
    a = max(a, __shfl_xor_sync(0xffffffffu, a, 2));
    const bool nan_block = a >= 0x7f800000u, valid = vec < p.vecs;
    // floor(log2 amax) - emax + 127, at least 0 (amax 0 and subnormals too); 254 at most
    const uint32_t code = static_cast<uint32_t>(max(static_cast<int>(a >> 23) - Fmt<FMT>::emax, 0));
    encode8<FMT, SR>(p, static_cast<uint64_t>(row) * p.cols / 8 * Fmt<FMT>::bits + vec * Fmt<FMT>::bits,
                     static_cast<uint64_t>(row) * p.cols + 8ull * vec, y, code, valid, nan_block);
    const uint32_t s = nan_block ? 0xffu : code, lane = threadIdx.x & 15u;
    if (p.word_scales) {
        uint32_t w = s | (__shfl_down_sync(0xffffffffu, s, 4, 16) << 8);
        w |= __shfl_down_sync(0xffffffffu, w, 8, 16) << 16;
        if (p.sl == SL_MMA_X4) w = __shfl_sync(0xffffffffu, w, 0, 16);
        if ((vec | 15u) < p.vecs) {
            uint32_t off = row_at;
            if (p.sl == SL_MMA_X4) off += (vec >> 4) * 2048u + 512u * lane;      // lanes 0..3 write the four copies
            else off += p.sl == SL_MMA ? (vec >> 4) * 512u : vec >> 2;
            if (lane < (p.sl == SL_MMA_X4 ? 4u : 1u) && in_bounds(off, 4, p.scales_cap))
                *reinterpret_cast<uint32_t *>(p.scales + off) = w;
            return;
        }
    }
    if (valid && (vec & 3u) == 0)
        put_scale(p.scales, p.sl, static_cast<uint32_t>(row), vec >> 2, p.k_blocks, p.k_groups, s, p.scales_cap);
}

// The casts that a kernel is made for: one format, or a choice of formats at run
// time (six code bits and INT8, which few programs take; stochastic rounding).
enum Cast { NO_CAST, TO_E4M3, TO_E5M2, TO_E2M1, TO_OTHERS, STOCHASTIC };

template <int CAST>
__device__ __forceinline__ void cast_as(const NormParams &p, int64_t row, uint32_t row_at, uint32_t vec, const f2 (&y)[4]) {
    constexpr bool SR = CAST == STOCHASTIC;
    if (CAST == TO_E4M3) return cast8<MX_E4M3, false>(p, row, row_at, vec, y);
    if (CAST == TO_E5M2) return cast8<MX_E5M2, false>(p, row, row_at, vec, y);
    if (CAST == TO_E2M1) return cast8<MX_E2M1, false>(p, row, row_at, vec, y);
    switch (p.fmt) {
        case MX_E2M3: return cast8<MX_E2M3, SR>(p, row, row_at, vec, y);
        case MX_E3M2: return cast8<MX_E3M2, SR>(p, row, row_at, vec, y);
        case MX_INT8: return cast8<MX_INT8, SR>(p, row, row_at, vec, y);
    }
    if (!SR) return;
    switch (p.fmt) {
        case MX_E4M3: return cast8<MX_E4M3, SR>(p, row, row_at, vec, y);
        case MX_E5M2: return cast8<MX_E5M2, SR>(p, row, row_at, vec, y);
        case MX_E2M1: return cast8<MX_E2M1, SR>(p, row, row_at, vec, y);
    }
}

// Rows blockIdx.x, blockIdx.x + gridDim.x, ...; a thread holds V vectors of
// eight values, vector i of thread t being i * blockDim + t (so four
// neighbouring lanes hold a block), and the weight's of the same columns.
// Vectors past the row's end are zero, like their weights, and not stored.
// Memory bounds it: a bf16 row with a residual moves 4 bytes a value in, 2 of h
// out, and 2 of y or 1 + 1/32 of E4M3 codes.  Measured (16384 x 4096 bf16):
// 88 us, 6.1 TB/s, with y, and 83 us, 5.7 TB/s, with codes (a copy makes 6.5);
// 8192 x 4096 fp32 with codes 73 us, 6.0 TB/s; one row of 4096 1.8 us, a chain
// of latencies.  Other casts of 16384 x 4096 bf16 (us; a copy of their bytes 67 to
// 72): E2M1 77, E2M3 82, E3M2 82, INT8 92; stochastic rounding E4M3 85, E2M1 88,
// E2M3 90, INT8 111.
template <bool BF16, bool RES, int V, int T, int CAST>
__global__ void __launch_bounds__(T, 1) norm_kernel(const __grid_constant__ NormParams p) {
    // the next row's loads are in flight while this one is worked on, where registers allow
    constexpr bool AHEAD = V * (BF16 ? 1 : 2) <= 4 && T <= 512;
    constexpr bool WIDE = V <= 2;                              // h stays widened between its two uses
    constexpr int SIZE = BF16 ? 2 : 4;
    after_predecessor();
    __shared__ __align__(16) float red[2][32];
    Raw<BF16> x[AHEAD ? V : 1], r[AHEAD && RES ? V : 1];
    f2 w[AHEAD ? V : 1][4];
    const uint32_t t = threadIdx.x, n = blockDim.x;
    const int64_t first = blockIdx.x, step = gridDim.x;
    // this thread's first vector of the row to be fetched, and of the row worked on
    const char *px = static_cast<const char *>(p.x) + (first * p.ldx + 8 * t) * SIZE;
    const char *pr = RES ? static_cast<const char *>(p.res) + (first * p.ldr + 8 * t) * SIZE : nullptr;
    char *ph = RES ? static_cast<char *>(p.h) + (first * p.ldh + 8 * t) * SIZE : nullptr;
    char *py = p.y ? static_cast<char *>(p.y) + (first * p.ldy + 8 * t) * SIZE : nullptr;
    auto fetch = [&] {
#pragma unroll
        for (int i = 0; AHEAD && i < V; ++i) {
            if (i * n + t >= p.vecs) continue;
            x[AHEAD ? i : 0].load(px, static_cast<int64_t>(i * n) * 8, p.wide);
            if (RES) r[AHEAD && RES ? i : 0].load(pr, static_cast<int64_t>(i * n) * 8, p.wide);
        }
        px += step * p.ldx * SIZE;
        if (RES) pr += step * p.ldr * SIZE;
    };
    if (AHEAD) {
#pragma unroll
        for (int i = 0; i < V; ++i) {
            x[AHEAD ? i : 0].zero();
            if (RES) r[AHEAD && RES ? i : 0].zero();
        }
        fetch();
#pragma unroll
        for (int i = 0; i < V; ++i) {
#pragma unroll
            for (int j = 0; j < 4; ++j) w[AHEAD ? i : 0][j] = 0;
            if (i * n + t < p.vecs) load_weight8(p.w, p.w_f32, 8 * (i * n + t), w[AHEAD ? i : 0]);
        }
    }
    clear_sums(red);
    int turn = 0;
    for (int64_t row = first; row < p.rows; row += step, turn ^= 1) {
        Raw<BF16> h[V];
        if (!AHEAD) {
#pragma unroll
            for (int i = 0; i < V; ++i) {
                h[i].zero();
                if (i * n + t >= p.vecs) continue;
                h[i].load(px, static_cast<int64_t>(i * n) * 8, p.wide);
                if (RES) {
                    Raw<BF16> a;
                    a.load(pr, static_cast<int64_t>(i * n) * 8, p.wide);
                    h[i].add(a);
                }
            }
            px += step * p.ldx * SIZE;
            if (RES) pr += step * p.ldr * SIZE;
        }
#pragma unroll
        for (int i = 0; AHEAD && i < V; ++i) {
            h[i] = x[AHEAD ? i : 0];
            if (RES) h[i].add(r[AHEAD && RES ? i : 0]);
        }
        if (AHEAD && row + step < p.rows) fetch();
        f2 sq = 0, wide[WIDE ? V : 1][4];
#pragma unroll
        for (int i = 0; i < V; ++i) {
            if (RES && i * n + t < p.vecs) h[i].store(ph, static_cast<int64_t>(i * n) * 8, p.wide);
            f2 v[4];
            h[i].widen(v);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                sq = fma2(v[j], v[j], sq);
                if (WIDE) wide[WIDE ? i : 0][j] = v[j];
            }
        }
        if (RES) ph += step * p.ldh * SIZE;
        float s0, s1;
        unpair(sq, s0, s1);
        const float ss = cta_sum(s0 + s1, red[turn]);
        const float rstd = __frsqrt_rn(ss * p.inv_cols + p.eps);
        if (p.rstd && t == 0) p.rstd[row] = rstd;
        const f2 rstd2 = pair(rstd, rstd);
        const uint32_t r32 = static_cast<uint32_t>(row);
        const uint32_t row_at = p.sl == SL_PLAIN ? r32 * p.k_blocks
                                                 : (r32 >> 7) * p.k_groups * (p.sl == SL_MMA ? 512u : 2048u) +
                                                       ((r32 & 31u) << 4) + (((r32 >> 5) & 3u) << 2);
#pragma unroll
        for (int i = 0; i < V; ++i) {
            f2 y[4], wl[4] = {0, 0, 0, 0};
            if (!AHEAD && i * n + t < p.vecs) load_weight8(p.w, p.w_f32, 8 * (i * n + t), wl);
            if (!WIDE) h[i].widen(y);
#pragma unroll
            for (int j = 0; j < 4; ++j) y[j] = mul2(mul2(WIDE ? wide[WIDE ? i : 0][j] : y[j], rstd2), AHEAD ? w[AHEAD ? i : 0][j] : wl[j]);
            if (CAST != NO_CAST) cast_as<CAST>(p, row, row_at, i * n + t, y);
            if (p.y && i * n + t < p.vecs) {
                Raw<BF16> o;
                o.narrow(y);
                o.store(py, static_cast<int64_t>(i * n) * 8, p.wide);
            }
        }
        if (p.y) py += step * p.ldy * SIZE;
    }
}

struct BackParams {
    const void *dy, *h, *dres;
    int64_t rows, lddy, ldh, lddres, lddx;
    uint32_t cols, pieces;     // 16-byte pieces of a row
    const void *w;
    int w_f32;
    const float *rstd;
    void *dx;
    float *dw, *part;
    uint32_t parts;
    float inv_cols;
    uint32_t cluster, each;    // CTAs that share a row, and the pieces of each (the last has the rest)
    uint32_t threads, groups;  // threads to a CTA's share of a row, rows of a CTA at a time
    int stages;                // rows in each group's ring
};

// 16 bytes as loaded, eight bf16 values or four fp32 ones.
template <bool BF16> struct Piece {
    static constexpr int PAIRS = BF16 ? 4 : 2, VALUES = 2 * PAIRS;
    uint4 v;

    __device__ __forceinline__ void widen(f2 (&f)[PAIRS]) const {
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < PAIRS; ++i)
            f[i] = BF16 ? pair(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u))
                        : pair(__uint_as_float(w[2 * (i & 1)]), __uint_as_float(w[2 * (i & 1) + 1]));
    }
    __device__ __forceinline__ void narrow(const f2 (&f)[PAIRS]) {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < PAIRS; ++i) {
            float lo, hi;
            unpair(f[i], lo, hi);
            if (BF16) {
                w[i] = pack_bf16(lo, hi);
            } else {
                w[2 * (i & 1)] = __float_as_uint(lo);
                w[2 * (i & 1) + 1] = __float_as_uint(hi);
            }
        }
        v = make_uint4(w[0], w[1], w[2], w[3]);
    }
    // the weights of the piece's columns from `col`
    static __device__ __forceinline__ void weights(const void *w, int w_f32, uint32_t col, f2 (&f)[PAIRS]) {
#pragma unroll
        for (int i = 0; i < PAIRS; ++i) {
            if (w_f32) {
                const float2 a = reinterpret_cast<const float2 *>(static_cast<const float *>(w) + col)[i];
                f[i] = pair(a.x, a.y);
            } else {
                const uint32_t a = reinterpret_cast<const uint32_t *>(static_cast<const uint16_t *>(w) + col)[i];
                f[i] = pair(__uint_as_float(a << 16), __uint_as_float(a & 0xffff0000u));
            }
        }
    }
};

// Sum over a group of `warps` warps in the fixed order of cta_sum; `barrier` is
// the group's own, `red` its place (with room for a multiple of four).
__device__ __forceinline__ float group_sum(float s, float *red, uint32_t warps, uint32_t warp, uint32_t barrier) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    if (warps == 1) return s;
    if ((threadIdx.x & 31) == 0) red[warp] = s;
    asm volatile("bar.sync %0, %1;" ::"r"(barrier), "r"(warps * 32) : "memory");
    float4 t = *reinterpret_cast<const float4 *>(red);
    for (uint32_t i = 4; i < warps; i += 4) {
        const float4 u = *reinterpret_cast<const float4 *>(red + i);
        t.x += u.x;
        t.y += u.y;
        t.z += u.z;
        t.w += u.w;
    }
    return (t.x + t.y) + (t.z + t.w);
}

// Sum over the cluster, in the CTAs' order; every thread has its CTA's sum s and
// gets the cluster's.  `all` is the same place in every CTA, and not the last
// row's: a CTA may still read that one.
__device__ __forceinline__ float cluster_sum(float s, float *all, uint32_t cluster, uint32_t rank) {
    if (threadIdx.x < cluster) *cg::this_cluster().map_shared_rank(all + rank, threadIdx.x) = s;
    cg::this_cluster().sync();
    s = all[0];
    for (uint32_t i = 1; i < cluster; ++i) s += all[i];
    return s;
}

// WIDE: a row is shared by the CTAs of a cluster, each with its own columns.
// Cluster b (else CTA b) takes rows b * groups to b * groups +
// groups - 1, group k of the CTA the kth, and every parts * groups rows from
// there; a thread has V pieces of its CTA's share of a row, piece i * threads + t.
// It keeps its columns' share of dweight in registers; at the end the groups'
// shares are added in order and written to part[b].
// The rows pass through a ring of p.stages rows in shared memory, where each
// thread copies its own columns ahead of their use and reads them twice (no
// other thread does, so the ring needs no barrier).  Registers for the next row
// instead: 51.5 us against 48 at 8192 x 4096 bf16; rows read twice from global
// memory: 308.
// Memory bounds it: dy, h and dres in, dx out, 8 bytes a bf16 value, and behind
// that the wait for each row's sum.  Measured, dweight's kernel of 3 to 4 us
// included: 16384 x 4096 bf16 85 us, 6.3 TB/s; 8192 x 4096 bf16 49 us, 5.5 TB/s,
// and fp32 85 us, 6.3 TB/s.
template <bool BF16, bool RES, int V, bool WIDE>
__global__ void __launch_bounds__(512, 1) norm_backward_kernel(const __grid_constant__ BackParams p) {
    using P = Piece<BF16>;
    constexpr int ARRAYS = RES ? 3 : 2;
    after_predecessor();
    __shared__ __align__(16) float red[2][32];
    __shared__ float across[WIDE ? 2 : 1][4];
    extern __shared__ __align__(16) uint4 ring[];              // [group][stage][array][piece]
    const uint32_t n = p.threads, group = threadIdx.x / n, t = threadIdx.x - group * n;
    const uint32_t warps = n / 32, warp = t >> 5, row_vecs = V * n, stage_vecs = ARRAYS * row_vecs;
    const uint32_t rank = WIDE ? blockIdx.x % p.cluster : 0u, block = WIDE ? blockIdx.x / p.cluster : blockIdx.x;
    const uint32_t base = rank * p.each, pieces = WIDE ? min(p.each, p.pieces - base) : p.pieces;    // of this CTA
    const int64_t first = static_cast<int64_t>(block) * p.groups + group, step = static_cast<int64_t>(WIDE ? p.parts : gridDim.x) * p.groups;
    constexpr int SIZE = BF16 ? 2 : 4;
    const char *in[3] = {static_cast<const char *>(p.dy) + first * p.lddy * SIZE + 16 * (base + t),
                         static_cast<const char *>(p.h) + first * p.ldh * SIZE + 16 * (base + t),
                         RES ? static_cast<const char *>(p.dres) + first * p.lddres * SIZE + 16 * (base + t) : nullptr};
    const int64_t by[3] = {step * p.lddy * SIZE, step * p.ldh * SIZE, RES ? step * p.lddres * SIZE : 0};
    char *out = static_cast<char *>(p.dx) + first * p.lddx * SIZE + 16 * (base + t);
    uint4 *mine = ring + group * p.stages * stage_vecs + t;
    const uint32_t mine32 = static_cast<uint32_t>(__cvta_generic_to_shared(mine));
    auto fetch = [&](uint32_t at) {                            // the next row to be read
#pragma unroll
        for (int a = 0; a < ARRAYS; ++a) {
#pragma unroll
            for (int i = 0; i < V; ++i)
                if (i * n + t < pieces)
                    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(mine32 + (at + a * row_vecs + i * n) * 16),
                                 "l"(in[a] + i * n * 16)
                                 : "memory");
            in[a] += by[a];
        }
    };
    auto commit = [] { asm volatile("cp.async.commit_group;" ::: "memory"); };
    for (int s = 0; s < p.stages - 1; ++s) {
        if (first + s * step < p.rows) fetch(s * stage_vecs);
        commit();
    }
    f2 acc[V][P::PAIRS], w[V][P::PAIRS];
#pragma unroll
    for (int i = 0; i < V; ++i) {
#pragma unroll
        for (int j = 0; j < P::PAIRS; ++j) acc[i][j] = 0;
        if (i * n + t < pieces) P::weights(p.w, p.w_f32, (base + i * n + t) * P::VALUES, w[i]);
    }
    clear_sums(red);
    if (WIDE) cg::this_cluster().sync();              // the others run: their shared memory can be written
    float rstd = first < p.rows ? p.rstd[first] : 0.0f;
    int turn = 0;
    const uint32_t last = (p.stages - 1) * stage_vecs, place = group * ((warps + 3) & ~3u);
    uint32_t at = 0;
    for (int64_t row = first; row < p.rows; row += step, turn ^= 1) {
        const f2 rs = pair(rstd, rstd);
        if (row + step < p.rows) rstd = p.rstd[row + step];
        // this thread's copies of the row have landed (all but the last stages - 2 groups)
        if (p.stages == 2) asm volatile("cp.async.wait_group 0;" ::: "memory");
        else if (p.stages == 3) asm volatile("cp.async.wait_group 1;" ::: "memory");
        else asm volatile("cp.async.wait_group 2;" ::: "memory");
        if (row + (p.stages - 1) * step < p.rows) fetch(at == 0 ? last : at - stage_vecs);
        commit();
        auto get = [&](int a, int i, P &x) { x.v = mine[at + a * row_vecs + i * n]; };
        // the piece's a = dy * weight and n = h * rstd, and dy
        auto terms = [&](int i, f2 (&a)[P::PAIRS], f2 (&nn)[P::PAIRS], f2 (&dy)[P::PAIRS]) {
            P g, h;
            get(0, i, g);
            get(1, i, h);
            g.widen(dy);
            h.widen(nn);
#pragma unroll
            for (int j = 0; j < P::PAIRS; ++j) {
                nn[j] = mul2(nn[j], rs);
                a[j] = mul2(dy[j], w[i][j]);
            }
        };
        f2 dot = 0;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            if (i * n + t >= pieces) continue;
            f2 a[P::PAIRS], nn[P::PAIRS], dy[P::PAIRS];
            terms(i, a, nn, dy);
#pragma unroll
            for (int j = 0; j < P::PAIRS; ++j) {
                acc[i][j] = fma2(dy[j], nn[j], acc[i][j]);
                dot = fma2(a[j], nn[j], dot);
            }
        }
        float s0, s1;
        unpair(dot, s0, s1);
        float c = group_sum(s0 + s1, red[turn] + place, warps, warp, 1 + group);
        if (WIDE) c = cluster_sum(c, across[WIDE ? turn : 0], p.cluster, rank);
        c *= p.inv_cols;
        const f2 minus_c = pair(-c, -c);
#pragma unroll
        for (int i = 0; i < V; ++i) {
            if (i * n + t >= pieces) continue;
            f2 a[P::PAIRS], nn[P::PAIRS], dy[P::PAIRS];
            terms(i, a, nn, dy);
#pragma unroll
            for (int j = 0; j < P::PAIRS; ++j) a[j] = mul2(rs, fma2(nn[j], minus_c, a[j]));
            P o;
            if (RES) {
                get(2, i, o);
                o.widen(nn);
#pragma unroll
                for (int j = 0; j < P::PAIRS; ++j) a[j] = add2(a[j], nn[j]);
            }
            o.narrow(a);
            *reinterpret_cast<uint4 *>(out + i * n * 16) = o.v;
        }
        out += step * p.lddx * SIZE;
        at = at == last ? 0 : at + stage_vecs;
    }
    // the groups' shares, through the ring (its copies have landed) and in order
    float *part = p.part + static_cast<int64_t>(block) * p.cols;
    float *shares = reinterpret_cast<float *>(ring);
    if (p.groups > 1) {
        asm volatile("cp.async.wait_group 0;" ::: "memory");
        __syncthreads();
    }
#pragma unroll
    for (int i = 0; i < V; ++i) {
        if (i * n + t >= pieces) continue;
        float *to = (p.groups > 1 ? shares + group * p.cols : part) + (base + i * n + t) * P::VALUES;
#pragma unroll
        for (int j = 0; j < P::PAIRS; ++j) {
            float lo, hi;
            unpair(acc[i][j], lo, hi);
            reinterpret_cast<float2 *>(to)[j] = make_float2(lo, hi);
        }
    }
    if (p.groups == 1) return;
    __syncthreads();
    for (uint32_t c = threadIdx.x; c < p.cols; c += blockDim.x) {
        float s = shares[c];
        for (uint32_t k = 1; k < p.groups; ++k) s += shares[k * p.cols + c];
        part[c] = s;
    }
}

// dweight[c] = the sum of the parts: 32 columns to a CTA, warp w adds parts w,
// w + 32, ..., and the warps' sums are added in their order.  No atomics, so the
// result has one value; 296 parts x 4096 columns are 4.8 MB that the backward
// kernel has just left in L2.
constexpr int DW_WARPS = 32;
__global__ void __launch_bounds__(32 * DW_WARPS) norm_dweight_kernel(const float *part, uint32_t parts, uint32_t cols, float *dw) {
    __shared__ float red[DW_WARPS][32];
    const uint32_t lane = threadIdx.x & 31u, warp = threadIdx.x >> 5, c = blockIdx.x * 32 + lane;    // cols % 32 == 0
    after_predecessor();
    float s = 0.0f;
#pragma unroll 10
    for (uint32_t i = warp; i < parts; i += DW_WARPS) s += part[static_cast<int64_t>(i) * cols + c];
    red[warp][lane] = s;
    __syncthreads();
    if (warp != 0) return;
#pragma unroll
    for (int i = 1; i < DW_WARPS; ++i) s += red[i][lane];
    dw[c] = s;
}

// Launches a kernel that begins with after_predecessor().
template <typename Kern, typename... Args>
cudaError_t launch_early(Kern kern, unsigned grid, unsigned cluster, unsigned threads, size_t smem, cudaStream_t st,
                         const Args &...args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = cluster;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kern, args...);
}

int threads_for(uint32_t vecs, int v) { return static_cast<int>((vecs + v - 1) / v + 31) / 32 * 32; }

// CTAs of a kernel that the device runs at a time; asked for each launch shape
// (a few hundred nanoseconds on the host).
template <typename Kern>
int64_t resident(Kern kern, int threads, int sms) {
    int n = 0;
    return cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, kern, threads, 0) == cudaSuccess && n > 0 ? int64_t{n} * sms : sms;
}

template <bool BF16, bool RES, int V, int T, int CAST>
cudaError_t launch_norm(const NormParams &p, int sms, cudaStream_t st) {
    auto kern = norm_kernel<BF16, RES, V, T, CAST>;
    const int threads = threads_for(p.vecs, V);
    const int64_t most = p.rows <= sms ? p.rows : resident(kern, threads, sms);
    return launch_early(kern, static_cast<unsigned>(p.rows < most ? p.rows : most), 1, threads, 0, st, p);
}

template <bool BF16, bool RES, int V, int T>
cudaError_t launch_norm_cast(const NormParams &p, int cast, int sms, cudaStream_t st) {
    switch (cast) {
        case NO_CAST: return launch_norm<BF16, RES, V, T, NO_CAST>(p, sms, st);
        case TO_E4M3: return launch_norm<BF16, RES, V, T, TO_E4M3>(p, sms, st);
        case TO_E5M2: return launch_norm<BF16, RES, V, T, TO_E5M2>(p, sms, st);
        case TO_E2M1: return launch_norm<BF16, RES, V, T, TO_E2M1>(p, sms, st);
        case TO_OTHERS: return launch_norm<BF16, RES, V, T, TO_OTHERS>(p, sms, st);
        default: return launch_norm<BF16, RES, V, T, STOCHASTIC>(p, sms, st);
    }
}

// Vectors of a thread: a row stays in one warp while four vectors a thread hold
// it (its sum then needs no barrier), and takes about 256 threads beyond that,
// fp32 512 with two vectors (four take too many registers for the next row to
// be in flight).  Measured (with residual and E4M3 cast, us with V = 1, 2, 4):
//   vecs   32   32768 x 256  bf16   10.7  15.7  23.7
//   vecs   64   16384 x 512  bf16   11.1   9.8  14.4
//   vecs  128   16384 x 1024 bf16   21.2  22.2  19.9
//   vecs  132   1013 x 1056  fp32    4.5   5.3   5.9
//   vecs  256   16384 x 2048 bf16   42.2  43.9  44.0
//   vecs  512   16384 x 4096 bf16   82.4  82.9  84.7
//   vecs  512   8192 x 4096  fp32   78.2  73.5  90.3
//   vecs 1024   8192 x 8192  bf16         86.6  83.7
//   vecs 1024   8192 x 8192  fp32          148   179
// Wider rows have four vectors a thread: fp32 without the next row in flight and
// with one CTA to an SM (108 registers x 512 threads), 4096 x 16384 183, 4.8 TB/s
// (with y instead of codes 196, 5.5); bf16 in the same way beyond 512 threads, 2048 x
// 32768 88, 5.4 TB/s (91, 5.9).  At 1024 threads fp32 with a residual spills up to
// 40 bytes of its 64 registers.
template <bool BF16, bool RES>
cudaError_t launch_norm_v(const NormParams &p, int cast, int sms, cudaStream_t st) {
    const int v = p.vecs <= 32 ? 1 : p.vecs <= 64 ? 2 : p.vecs <= 128 ? 4 : p.vecs <= 256 ? 1 : p.vecs <= (BF16 ? 512 : 1024) ? 2 : 4;
    if (v == 1) return launch_norm_cast<BF16, RES, 1, 512>(p, cast, sms, st);
    if (v == 2) return launch_norm_cast<BF16, RES, 2, 512>(p, cast, sms, st);
    if (p.vecs <= 4 * 512) return launch_norm_cast<BF16, RES, 4, 512>(p, cast, sms, st);
    return launch_norm_cast<BF16, RES, 4, 1024>(p, cast, sms, st);
}

constexpr int BACK_SMEM = 226 * 1024;        // with the sums' 288 bytes, what a CTA can have
constexpr int BACK_HALF = 112 * 1024;        // two CTAs to an SM
constexpr uint32_t BACK_THREADS = 512, BACK_V = 4;

template <bool BF16, bool RES, int V, bool WIDE>
cudaError_t launch_back(const BackParams &p, cudaStream_t st) {
    static std::atomic<uint64_t> done{0};
    auto kern = norm_backward_kernel<BF16, RES, V, WIDE>;
    const cudaError_t e = ensure_smem_limit(kern, BACK_SMEM, done);
    if (e != cudaSuccess) return e;
    return launch_early(kern, p.parts * p.cluster, p.cluster, p.threads * p.groups,
                        p.groups * p.stages * (RES ? 3 : 2) * V * p.threads * 16, st, p);
}

// A row wider than the 2048 pieces that 512 threads of four hold is shared by a
// cluster of two or four CTAs.  Pieces of a thread: as many as leave a row a CTA
// of 256 threads, or several rows the threads of one.  Measured (us with V = 1,
// 2, 4):
//   pieces   32   32768 x 256  bf16   16.9  17.5  19.1
//   pieces   64   16384 x 512  bf16   18.2  16.8  16.2
//   pieces  128   16384 x 1024 bf16   30.7  28.6  28.7
//   pieces  264   333 x 1056   fp32    7.7   7.5   6.5
//   pieces  320   8192 x 2560  bf16   37.4  40.9  35.2
//   pieces  448   8192 x 3584  bf16   61.3  44.4  44.9
//   pieces  512   8192 x 4096  bf16   64.5  49.2  50.6
//   pieces 1024   4096 x 8192  bf16         58.1  51.8
// Threads of a CTA of several rows, 128, 256, 512 (and one row): 32768 x 256
// 21.6, 16.7, 20.1 (54); 16384 x 1024 33.2, 29.0, 30.9 (43).
// The ring has two to four rows of each group, in half of the shared memory if
// they fit there: two CTAs to an SM, 2 x 148 parts, hide each other's sums (one
// CTA: 8192 x 4096 59 us against 49).  Where the SM has one CTA at a time, more
// than 148 parts would run one after the other (2048 x 16384 65 us against 54);
// of clusters the device may hold somewhat fewer than 148 CTAs' worth.
// The parts decide dweight's bits, so they go by the three arrays that a row has
// with dres, also without it.  Where two rows of two arrays would still fit into
// half of the shared memory, the ring then has three (without dres, us with 296
// parts and two rows, 148 and two, three, four): 8192 x 10240 bf16 104.7, 97.2,
// 96.2, 98.1; 8192 x 5120 fp32 89.2, 85.8, 80.1, 80.3; 600 x 5120 fp32 15.9, 13.3,
// 12.9, 14.1; 4096 x 7168 fp32 62.2, 58.0, 61.2, 61.0.
template <bool BF16, bool RES>
cudaError_t launch_backward_v(BackParams &p, cudaStream_t st) {
    p.cluster = p.pieces <= BACK_V * BACK_THREADS ? 1 : p.pieces <= 2 * BACK_V * BACK_THREADS ? 2 : 4;    // cols <= 32768
    p.each = (p.pieces + p.cluster - 1) / p.cluster;
    const int v = p.pieces <= 32 ? 1 : p.pieces <= 384 || p.pieces > 512 ? 4 : 2;
    p.threads = threads_for(p.each, v);
    p.groups = std::max(1u, 256 / p.threads);
    const int array = p.groups * v * p.threads * 16, row = (RES ? 3 : 2) * array;     // bytes of a stage, 96 KB at most
    const bool one = 2 * 3 * array > BACK_HALF;                                     // CTA to an SM
    p.stages = one && 2 * row <= BACK_HALF ? 3 : std::max(2, std::min(4, BACK_HALF / row));
    if (p.cluster > 1) p.parts = std::min(p.parts, p.cluster == 2 ? 72u : 32u);
    else if (one) p.parts = std::min(p.parts, 148u);
    p.parts = static_cast<uint32_t>(std::min<int64_t>((p.rows + p.groups - 1) / p.groups, p.parts));
    if (p.cluster > 1) return launch_back<BF16, RES, 4, true>(p, st);
    if (v == 1) return launch_back<BF16, RES, 1, false>(p, st);
    if (v == 2) return launch_back<BF16, RES, 2, false>(p, st);
    return launch_back<BF16, RES, 4, false>(p, st);
}

}  // namespace mxnorm

cudaError_t mx_launch_rmsnorm(const MxNormArgs &a, cudaStream_t st) {
    using namespace mxnorm;
    NormParams p;
    p.x = a.x; p.res = a.residual; p.rows = a.rows; p.ldx = a.ldx; p.ldr = a.ldr; p.ldh = a.ldh; p.ldy = a.ldy;
    p.cols = static_cast<uint32_t>(a.cols);
    p.vecs = p.cols / 8;
    p.w = a.weight; p.w_f32 = a.wdt == MX_F32; p.eps = a.eps;
    p.inv_cols = 1.0f / static_cast<float>(a.cols);
    p.h = a.h; p.y = a.y; p.rstd = a.rstd;
    p.codes = static_cast<uint8_t *>(a.codes); p.scales = static_cast<uint8_t *>(a.scales);
    p.fmt = a.fmt; p.sl = a.sl;
    p.key = fmix32_host(static_cast<uint32_t>(a.seed)) ^ static_cast<uint32_t>(a.seed >> 32);
    p.k_blocks = p.cols / 32;
    p.k_groups = (p.k_blocks + 3) / 4;
    p.codes_cap = a.codes ? mx_codes_bytes(static_cast<mx_fmt>(a.fmt), a.rows, a.cols) : 0;
    p.scales_cap = a.codes ? mx_scales_bytes(static_cast<mx_scale_layout>(a.sl), a.rows, a.cols) : 0;
    const int cast = !a.codes ? NO_CAST
                     : a.rnd == MX_SR ? STOCHASTIC
                     : a.fmt == MX_E4M3 ? TO_E4M3
                     : a.fmt == MX_E5M2 ? TO_E5M2
                     : a.fmt == MX_E2M1 ? TO_E2M1
                                        : TO_OTHERS;
    auto on32 = [](const void *q, int64_t ld) { return !q || ((reinterpret_cast<uintptr_t>(q) | static_cast<uintptr_t>(ld * 4)) & 31u) == 0; };
    p.wide = on32(a.x, a.ldx) && on32(a.residual, a.ldr) && on32(a.h, a.ldh) && on32(a.y, a.ldy);
    p.word_scales = (reinterpret_cast<uintptr_t>(a.scales) & 3u) == 0 && (a.sl != MX_SCALES_PLAIN || p.k_blocks % 4 == 0);
    if (a.xdt == MX_BF16) return p.res ? launch_norm_v<true, true>(p, cast, a.num_sms, st) : launch_norm_v<true, false>(p, cast, a.num_sms, st);
    return p.res ? launch_norm_v<false, true>(p, cast, a.num_sms, st) : launch_norm_v<false, false>(p, cast, a.num_sms, st);
}

cudaError_t mx_launch_rmsnorm_backward(const MxNormBackArgs &a, cudaStream_t st) {
    using namespace mxnorm;
    BackParams p;
    p.dy = a.dy; p.h = a.h; p.dres = a.dres; p.rows = a.rows;
    p.lddy = a.lddy; p.ldh = a.ldh; p.lddres = a.lddres; p.lddx = a.lddx;
    p.cols = static_cast<uint32_t>(a.cols);
    p.pieces = p.cols / (a.xdt == MX_BF16 ? 8 : 4);
    p.w = a.weight; p.w_f32 = a.wdt == MX_F32; p.rstd = a.rstd;
    p.dx = a.dx; p.dw = a.dweight; p.part = a.part; p.parts = static_cast<uint32_t>(a.parts);
    p.inv_cols = 1.0f / static_cast<float>(a.cols);
    const cudaError_t e = a.xdt == MX_BF16 ? (p.dres ? launch_backward_v<true, true>(p, st) : launch_backward_v<true, false>(p, st))
                                           : (p.dres ? launch_backward_v<false, true>(p, st) : launch_backward_v<false, false>(p, st));
    if (e != cudaSuccess) return e;
    return launch_early(norm_dweight_kernel, p.cols / 32, 1, 32 * DW_WARPS, 0, st, static_cast<const float *>(p.part), p.parts,
                        p.cols, p.dw);
}

int mx_read_norm_bounds_status() {
    int b = 0;
    if (cudaMemcpyFromSymbol(&b, mxk::g_bounds_status, sizeof(int)) != cudaSuccess) return MX_ERR_CUDA;
    const int zero = 0;
    if (cudaMemcpyToSymbol(mxk::g_bounds_status, &zero, sizeof(int)) != cudaSuccess) return MX_ERR_CUDA;
    return b;
}
