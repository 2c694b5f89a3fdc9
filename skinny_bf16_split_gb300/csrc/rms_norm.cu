// rms_norm.cu -- RMS norm with the residual's addition and an 8-bit output, and
// the 8-bit quantisation of rows without a norm.
//
//     h = bf16(x + r);  y = h * rstd * w,  rstd = 1 / sqrt(mean(h^2) + eps)
//
// One pass over memory: a row (or, for up to 1024 columns, a warp's row) stays
// in registers between the reduction and the store.  The quantised values do
// not depend on rstd: with p = h * w, int8 q = rint(127 p / max|p|), so one
// reduction gives the sum of squares and max|p| together.
//
// Exact rounding.  h and w have 8 significant bits, so p is exact in FP32 (16
// bits), and so are 127 p (23) and 448 p (19).
//   int8: the quotient's nearest integer guess c = rint(127 p * (1 / P)) is
//     settled by the remainder 127 p - c P, which FP32 holds exactly (7 + 16
//     bits): compare twice its size with P, ties to even.
//   e4m3: a quotient that is no tie (of 5 bits) differs from every tie by at
//     least 2^-21 of itself (the integers 448 p 2^s and tie * P differ by one or
//     more, and tie * P < 2^21), more than the 2^-23 of a product with a rounded
//     reciprocal; one Newton step makes a quotient that is a tie exact, and the
//     conversion then rounds ties to even.
// P below 2^-100 is flushed (stored as zero), which keeps 1 / P finite.  P and the 127 or 448 are both
// taken times 2^-10, so that neither 448 p nor 1 / P leaves FP32's range for p up to 2^128.  At the
// other end, P = 2^-100, that is exact for every p whose quotient does not round to zero (p > 2^-119),
// the remainder 127 p - c P too; e4m3's is rounded at 2^-149, 2^-6 of itself at most.
//
// Bound: DRAM.  Bytes of a row: 2 cols (x) + 4 cols with a residual + the output.  Measured
// with a residual, of the copy rate: 8192 x 7168 to BF16 68.4 us (101 %), to int8 66.7 (91 %), to
// e4m3 64.2 (95 %); 8192 x 7161, every row misaligned, to BF16 95.5 (72 %); one row 2.9 us.
// Rows of more than 16384 columns have 64 or 72 elements a thread, of which 0.3 to 2.1 KB spill: 200 x 40000 to int8
// 28 us (30 %).
#include <cuda_bf16.h>

#include "internal.h"
#include "layer.h"

namespace dep {
namespace {

struct NormParams {
    const uint16_t *x, *r, *w;
    uint16_t *h;
    void *out;
    float *scale;
    int64_t xs, rs, hs, os;
    int64_t rows;
    int32_t cols;
    float eps;
};

constexpr float kTiny = 0x1p-100f;
constexpr float kDown = 0x1p-10f;  // of P, 127 and 448 in the quotients

__device__ __forceinline__ float bf(uint32_t bits16) { return __uint_as_float(bits16 << 16); }

// Largest value; a NaN on either side gives a NaN.
__device__ __forceinline__ float max_nan(float a, float b)
{
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

// Rows that are not aligned, or not whole vectors (VEC false).  A thread's eight elements
// start where a granule of x's row starts, so contiguous matrices with any number of columns,
// whose rows are all misaligned alike, are still moved in whole granules, all but the row's
// ends.  A tensor aligned otherwise (the weight, a view) is loaded as the two granules that
// hold the eight elements, and shifted; it is stored as the granule that the eight start in,
// whose first elements come from the lane before.  (e4m3: a thread's elements start at a
// multiple of eight, so that they belong to one group.)  What granules at the ends of a warp
// or row would take from outside goes element by element.

// Words [s / 2, s / 2 + 4) (in 16-bit steps s <= 8) of the eight words a, b.
__device__ __forceinline__ uint4 shift16(uint4 a, uint4 b, int s)
{
    if (s & 8)
        return b;
    uint32_t w[7] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z};
    if (s & 4) {
        w[0] = a.z, w[1] = a.w, w[2] = b.x, w[3] = b.y, w[4] = b.z, w[5] = b.w;
    }
    if (s & 2) {
#pragma unroll
        for (int i = 0; i < 5; ++i)
            w[i] = w[i + 1];
    }
    if (s & 1) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            w[i] = __funnelshift_r(w[i], w[i + 1], 16);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// Eight consecutive elements (16 bits each) from column c on; columns outside 0..n-1 read as zero.
template <bool VEC>
__device__ __forceinline__ uint4 load8(const uint16_t *p, int c, int n)
{
    if (VEC)
        return c < n ? *reinterpret_cast<const uint4 *>(p + c) : make_uint4(0, 0, 0, 0);
    const int s = (int)((reinterpret_cast<uintptr_t>(p) >> 1) + c) & 7;
    const uint4 *g = reinterpret_cast<const uint4 *>(p + c - s);
    if (s == 0 && c >= 0 && c + 8 <= n)
        return *g;
    if (c >= s && c - s + 16 <= n)
        return shift16(g[0], g[1], s);
    uint32_t v[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int e = c + 2 * i;
        const uint32_t lo = e >= 0 && e < n ? p[e] : 0, hi = e + 1 >= 0 && e + 1 < n ? p[e + 1] : 0;
        v[i] = lo | hi << 16;
    }
    return make_uint4(v[0], v[1], v[2], v[3]);
}

// Store them; every lane of the warp calls, with consecutive c.
template <bool VEC>
__device__ __forceinline__ void store8(uint16_t *p, int c, int n, uint4 v)
{
    if (VEC) {
        if (c < n)
            *reinterpret_cast<uint4 *>(p + c) = v;
        return;
    }
    const int s = (int)((reinterpret_cast<uintptr_t>(p) >> 1) + c) & 7, lane = threadIdx.x & 31;
    uint4 out = v;
    if (s) {  // the same for all lanes
        uint4 before;
        before.x = __shfl_up_sync(~0u, v.x, 1);
        before.y = __shfl_up_sync(~0u, v.y, 1);
        before.z = __shfl_up_sync(~0u, v.z, 1);
        before.w = __shfl_up_sync(~0u, v.w, 1);
        out = shift16(before, v, 8 - s);
    }
    const bool own = (lane > 0 || s == 0) && c >= s && c - s + 8 <= n;  // this lane stores its first granule whole
    const bool next = s == 0 || (lane < 31 && c + 8 >= s && c + 16 - s <= n);  // and the next lane the one after
    if (own)
        *reinterpret_cast<uint4 *>(p + c - s) = out;
    const uint32_t a[4] = {v.x, v.y, v.z, v.w};
    if (!own || !next)
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (c + i >= 0 && c + i < n && !(i < 8 - s ? own : next))
                p[c + i] = (uint16_t)(a[i / 2] >> (16 * (i & 1)));
}

// The same for eight bytes in granules of eight.
template <bool VEC>
__device__ __forceinline__ void store8b(uint8_t *p, int c, int n, uint2 v)
{
    if (VEC) {
        if (c < n)
            *reinterpret_cast<uint2 *>(p + c) = v;
        return;
    }
    const int s = (int)(reinterpret_cast<uintptr_t>(p) + c) & 7, lane = threadIdx.x & 31;
    const uint64_t mine = (uint64_t)v.y << 32 | v.x;
    uint64_t out = mine;
    if (s) {
        const uint64_t before = __shfl_up_sync(~0u, (unsigned long long)mine, 1);
        out = before >> (64 - 8 * s) | mine << (8 * s);
    }
    const bool own = (lane > 0 || s == 0) && c >= s && c - s + 8 <= n;
    const bool next = s == 0 || (lane < 31 && c + 8 >= s && c + 16 - s <= n);
    if (own)
        *reinterpret_cast<uint64_t *>(p + c - s) = out;
    if (!own || !next)
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (c + i >= 0 && c + i < n && !(i < 8 - s ? own : next))
                p[c + i] = (uint8_t)(mine >> (8 * i));
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi)
{
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

// rint(127 p / P) in the low byte, exactly (see above), from P times kDown; inv = 1 / that, rounded.  The guess is read
// off the mantissa of its sum with 1.5 * 2^23 (conversions run at an eighth of the rate of an
// addition).  P infinite and inv zero (a flushed row): zero.
__device__ __forceinline__ uint32_t quant_int8(float p, float P, float inv)
{
    const float t = 127.0f * kDown * p, u = fmaf(t, inv, 12582912.0f);
    const float rem = fmaf(-(u - 12582912.0f), P, t), two = fabsf(rem) * 2.0f;
    const uint32_t c = __float_as_uint(u);
    const uint32_t step = rem > 0.0f ? 1u : 0xFFFFFFFFu;
    return two > P || (two == P && (c & 1)) ? c + step : c;
}

// 448 p / P to within far less than half an e4m3 step, exact where it is a tie; P and inv as above.
__device__ __forceinline__ float quot_e4m3(float p, float P, float inv)
{
    const float t = 448.0f * kDown * p;
    const float s = t * inv;
    return fmaf(fmaf(-s, P, t), inv, s);
}

__device__ __forceinline__ uint32_t pack_e4m3(float lo, float hi)
{
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}

// Whether the squares of a row leave FP32's range, by the 1 / rms that they gave: values of 2^56 or so and more or, with
// next to no eps, all below 2^-50.
__device__ __forceinline__ bool outside(float rstd) { return rstd == 0.0f || rstd > 0x1p50f; }

// Such a row: 1 / rms once more, of the row times a power of two, and what depends on it: BF16 values; scales, which
// have been stored as if it were one.  By memory and apart from the way of all other rows, whose registers
// it would take.  All threads of the row call.
template <int FMT, bool WARP_ROW>
__device__ __forceinline__ void norm_outside(const NormParams &a, uint32_t row, float rstd, float2 *part)
{
    const int t = threadIdx.x, threads = WARP_ROW ? 32 : blockDim.x, n = a.cols;
    const float f = rstd > 1.0f ? 0x1p80f : 0x1p-80f;
    const uint16_t *h = a.r ? a.h + row * a.hs : a.x + row * a.xs;
    if (WARP_ROW)
        __syncwarp();  // h is stored
    else
        __syncthreads();  // and the warps' first parts have been read
    float sum = 0.0f;
#pragma unroll 1
    for (int c = t; c < n; c += threads)
        sum = fmaf(bf(h[c]) * f, bf(h[c]) * f, sum);
#pragma unroll
    for (int o = 16; o; o >>= 1)
        sum += __shfl_xor_sync(~0u, sum, o);
    if (!WARP_ROW) {
        if ((t & 31) == 0)
            part[t >> 5].x = sum;
        __syncthreads();
        sum = 0.0f;
#pragma unroll 1
        for (int i = 0; i < threads / 32; ++i)
            sum += part[i].x;
    }
    const float r = f / sqrtf(sum / (float)n + a.eps * f * f);
    if (FMT == DEP_QUANT_NONE) {
        uint16_t *o = static_cast<uint16_t *>(a.out) + row * a.os;
#pragma unroll 1
        for (int c = t; c < n; c += threads)  // (o may be x: an element is read and written by one thread)
            o[c] = (uint16_t)pack_bf16(bf(h[c]) * (a.w ? bf(a.w[c]) : 1.0f) * r, 0.0f);
    } else {
        const int groups = FMT == DEP_QUANT_INT8 ? 1 : (n + DEP_QUANT_GROUP - 1) / DEP_QUANT_GROUP;
        float *scale = a.scale + (int64_t)row * groups;
        for (int i = t; i < groups; i += threads)
            if (scale[i] != 0.0f)  // zero: flushed
                scale[i] *= r;
    }
}

// WARP_ROW: blockDim = (32, 8), a row for each warp; else a row for each block of up to MAXT threads.
// Thread t holds the eight columns from 8 (t + i * threads) on, i < VPT, less c0 where rows are not aligned.
// Kernels held to 72 registers, as three blocks of 288 threads an SM would need.  BF16 rows that are not aligned: with 74
// the SM holds three blocks of seven warps instead of four, and 8192 x 7161 takes 108 us instead of 95.  Aligned e4m3
// rows: left to itself the compiler takes 64, and 8192 x 7168 65.1 us instead of 64.2.
template <int FMT, bool VEC, int MAXT>
constexpr bool held = MAXT == 256 && (VEC ? FMT == DEP_QUANT_E4M3 : FMT == DEP_QUANT_NONE);
template <int FMT, bool NORM, bool VEC, int VPT, bool WARP_ROW, int MAXT>
__global__ void __launch_bounds__(held<FMT, VEC, MAXT> ? 288 : MAXT, held<FMT, VEC, MAXT> ? 3 : 0)
    norm_kernel(const __grid_constant__ NormParams a)
{
    const uint32_t row = WARP_ROW ? blockIdx.x * 8 + threadIdx.y : blockIdx.x;
    if (WARP_ROW && row >= a.rows)
        return;
    const int t = threadIdx.x, threads = WARP_ROW ? 32 : blockDim.x, n = a.cols;
    const uint16_t *x = a.x + row * a.xs;
    const int c0 = VEC || FMT == DEP_QUANT_E4M3 ? 0 : (int)(reinterpret_cast<uintptr_t>(x) >> 1) & 7;
    uint4 hv[VPT], wv[VPT];
#pragma unroll
    for (int i = 0; i < VPT; ++i)
        hv[i] = load8<VEC>(x, 8 * (t + i * threads) - c0, n);
    if (NORM) {
        auto load_w = [&] {
#pragma unroll
            for (int i = 0; i < VPT; ++i)
                wv[i] = a.w ? load8<VEC>(a.w, 8 * (t + i * threads) - c0, n)
                            : make_uint4(0x3F803F80u, 0x3F803F80u, 0x3F803F80u, 0x3F803F80u);
        };
        // The weight's loads with the others where that pays: 8192 x 7168 to e4m3 66.5 -> 64.4 us, to BF16 69.8 ->
        // 68.8; but to int8 67.2 -> 83.1, and 8192 x 7161, with two granules for each vector, 94 -> 123.
        constexpr bool kEarly = VEC && VPT <= 4 && FMT != DEP_QUANT_INT8;
        if (kEarly)
            load_w();
        if (a.r) {
            const uint16_t *r = a.r + row * a.rs;
            uint4 rv[VPT];
#pragma unroll
            for (int i = 0; i < VPT; ++i)
                rv[i] = load8<VEC>(r, 8 * (t + i * threads) - c0, n);
#pragma unroll
            for (int i = 0; i < VPT; ++i) {
                uint32_t *h = &hv[i].x;
                const uint32_t *q = &rv[i].x;
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    h[j] = pack_bf16(bf(h[j] & 0xFFFFu) + bf(q[j] & 0xFFFFu), bf(h[j] >> 16) + bf(q[j] >> 16));
            }
        }
        if (!kEarly)
            load_w();
        if (a.r) {
            uint16_t *ho = a.h + row * a.hs;
#pragma unroll
            for (int i = 0; i < VPT; ++i)
                store8<VEC>(ho, 8 * (t + i * threads) - c0, n, hv[i]);
        }
    }
    // p = h * w of element j of vector i
    auto prod = [&](int i, int j) {
        const uint32_t h = (&hv[i].x)[j / 2];
        const float hf = bf(j & 1 ? h >> 16 : h & 0xFFFFu);
        if (!NORM)
            return hf;
        const uint32_t w = (&wv[i].x)[j / 2];
        return hf * bf(j & 1 ? w >> 16 : w & 0xFFFFu);
    };
    __shared__ float2 part[WARP_ROW ? 1 : MAXT / 32];
    float ss = 0.0f, top = 0.0f;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const uint32_t h = (&hv[i].x)[j / 2];
            const float hf = bf(j & 1 ? h >> 16 : h & 0xFFFFu);
            if (NORM)
                ss = fmaf(hf, hf, ss);
            if (FMT == DEP_QUANT_INT8)
                top = max_nan(top, fabsf(prod(i, j)));
        }
    }
    if (NORM || FMT == DEP_QUANT_INT8) {
#pragma unroll
        for (int o = 16; o; o >>= 1) {
            ss += __shfl_xor_sync(~0u, ss, o);
            if (FMT == DEP_QUANT_INT8)
                top = max_nan(top, __shfl_xor_sync(~0u, top, o));
        }
        if (!WARP_ROW) {
            if ((t & 31) == 0)
                part[t >> 5] = make_float2(ss, top);
            __syncthreads();
            if (MAXT <= 256) {  // every thread adds the warps' parts in the same order
                ss = 0.0f;
                top = 0.0f;
#pragma unroll
                for (int i = 0; i < MAXT / 32; ++i) {
                    const float2 v = i < threads / 32 ? part[i] : make_float2(0.0f, 0.0f);
                    ss += v.x;
                    if (FMT == DEP_QUANT_INT8)
                        top = max_nan(top, v.y);
                }
            } else {  // every warp adds them by the same shuffles
                const float2 v = (t & 31) < threads / 32 ? part[t & 31] : make_float2(0.0f, 0.0f);
                ss = v.x;
                top = v.y;
#pragma unroll
                for (int o = 16; o; o >>= 1) {
                    ss += __shfl_xor_sync(~0u, ss, o);
                    if (FMT == DEP_QUANT_INT8)
                        top = max_nan(top, __shfl_xor_sync(~0u, top, o));
                }
            }
        }
    }
    const float rstd = NORM ? 1.0f / sqrtf(ss / (float)n + a.eps) : 1.0f;
    // (squares outside FP32's range: BF16 rows are finished here, 8-bit rows, whose values do not depend on rms, below)
    if (NORM && FMT == DEP_QUANT_NONE && outside(rstd)) {
        norm_outside<FMT, WARP_ROW>(a, row, rstd, part);
        return;
    }
    const float per = NORM && outside(rstd) ? 1.0f : rstd;  // the scales' factor
    if (FMT == DEP_QUANT_NONE) {
        uint16_t *o = static_cast<uint16_t *>(a.out) + row * a.os;
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            uint4 v;
#pragma unroll
            for (int j = 0; j < 4; ++j)
                (&v.x)[j] = pack_bf16(prod(i, 2 * j) * rstd, prod(i, 2 * j + 1) * rstd);
            store8<VEC>(o, 8 * (t + i * threads) - c0, n, v);
        }
    } else if (FMT == DEP_QUANT_INT8) {
        const bool flush = top < kTiny;
        const float P = flush ? __int_as_float(0x7F800000) : top * kDown, inv = flush ? 0.0f : 1.0f / P;
        if (t == 0)
            a.scale[row] = flush ? 0.0f : top * per / 127.0f;
        uint8_t *o = static_cast<uint8_t *>(a.out) + row * a.os;
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            uint32_t v[2], b[8];
#pragma unroll
            for (int j = 0; j < 8; ++j)
                b[j] = quant_int8(prod(i, j), P, inv);
#pragma unroll
            for (int j = 0; j < 2; ++j)
                v[j] = __byte_perm(__byte_perm(b[4 * j], b[4 * j + 1], 0x0040), __byte_perm(b[4 * j + 2], b[4 * j + 3], 0x0040),
                                   0x5410);
            store8b<VEC>(o, 8 * (t + i * threads) - c0, n, make_uint2(v[0], v[1]));
        }
    } else {
        uint8_t *o = static_cast<uint8_t *>(a.out) + row * a.os;
        float *sc = a.scale + (int64_t)row * ((n + DEP_QUANT_GROUP - 1) / DEP_QUANT_GROUP);
#pragma unroll
        for (int i = 0; i < VPT; ++i) {  // 16 neighbouring threads hold a group
            const int c = 8 * (t + i * threads);
            float g = 0.0f;
#pragma unroll
            for (int j = 0; j < 8; ++j)
                g = max_nan(g, fabsf(prod(i, j)));
#pragma unroll
            for (int d = 8; d; d >>= 1)
                g = max_nan(g, __shfl_xor_sync(~0u, g, d));
            const bool flush = g < kTiny;
            const float P = g * kDown, inv = flush ? 0.0f : 1.0f / P;
            if ((t & 15) == 0 && c < n)
                sc[c / DEP_QUANT_GROUP] = flush ? 0.0f : g * per / 448.0f;
            uint32_t v[2] = {0, 0};
#pragma unroll
            for (int j = 0; j < 4; ++j)
                v[j / 2] |= pack_e4m3(quot_e4m3(prod(i, 2 * j), P, inv), quot_e4m3(prod(i, 2 * j + 1), P, inv))
                            << (16 * (j & 1));
            store8b<VEC>(o, c, n, make_uint2(v[0], v[1]));
        }
    }
    if (NORM && FMT != DEP_QUANT_NONE && outside(rstd))
        norm_outside<FMT, WARP_ROW>(a, row, rstd, part);
}

template <int FMT, bool NORM, bool VEC>
cudaError_t norm_launch(const NormParams &a, cudaStream_t s)
{
    const int vecs = (a.cols + (VEC ? 7 : 14)) / 8;  // with what a row's first granule may start before it
    const dim3 warp_grid((unsigned)((a.rows + 7) / 8)), grid((unsigned)a.rows), warps(32, 8);
    const auto threads = [&](int vpt) { return dim3((unsigned)(((vecs + vpt - 1) / vpt + 31) / 32 * 32)); };
    // A row for each warp up to 1024 columns; above, a row for each block, with just enough threads.
    if (vecs <= 32)
        norm_kernel<FMT, NORM, VEC, 1, true, 256><<<warp_grid, warps, 0, s>>>(a);
    else if (vecs <= 64)
        norm_kernel<FMT, NORM, VEC, 2, true, 256><<<warp_grid, warps, 0, s>>>(a);
    else if (vecs <= 128)
        norm_kernel<FMT, NORM, VEC, 4, true, 256><<<warp_grid, warps, 0, s>>>(a);
    else if (vecs <= 1024)
        norm_kernel<FMT, NORM, VEC, 4, false, 256><<<grid, threads(4), 0, s>>>(a);
    else if (vecs <= 2048)
        norm_kernel<FMT, NORM, VEC, 4, false, 512><<<grid, threads(4), 0, s>>>(a);
    else {
        constexpr int kMost = VEC ? 8 : 9;  // 65536 columns and a first granule that starts before them
        norm_kernel<FMT, NORM, VEC, kMost, false, 1024><<<grid, threads(kMost), 0, s>>>(a);
    }
    return cudaGetLastError();
}

template <bool VEC>
cudaError_t norm_dispatch(const NormParams &a, int quant, bool norm, cudaStream_t s)
{
    if (!norm)
        return quant == DEP_QUANT_INT8 ? norm_launch<DEP_QUANT_INT8, false, VEC>(a, s)
                                       : norm_launch<DEP_QUANT_E4M3, false, VEC>(a, s);
    return quant == DEP_QUANT_NONE   ? norm_launch<DEP_QUANT_NONE, true, VEC>(a, s)
           : quant == DEP_QUANT_INT8 ? norm_launch<DEP_QUANT_INT8, true, VEC>(a, s)
                                     : norm_launch<DEP_QUANT_E4M3, true, VEC>(a, s);
}

dep_status_t norm_entry(const dep_norm_args_t *p, bool norm, void *stream)
{
    if (!p || p->rows < 0 || p->cols < 1 || p->quant < DEP_QUANT_NONE || p->quant > DEP_QUANT_E4M3)
        return DEP_ERR_INVALID_ARG;
    const bool q8 = p->quant != DEP_QUANT_NONE;
    if (norm ? !(p->eps >= 0.0f) || (p->residual != nullptr) != (p->residual_out != nullptr)
             : p->residual || p->weight || p->residual_out || !q8)
        return DEP_ERR_INVALID_ARG;
    if (p->rows == 0)
        return DEP_OK;
    if (!p->x || !p->out || q8 != (p->scale != nullptr))
        return DEP_ERR_INVALID_ARG;
    if (p->cols > DEP_NORM_MAX_COLS || p->rows > INT32_MAX)
        return DEP_ERR_UNSUPPORTED;
    const int64_t C = p->cols, R = p->rows;
    if (p->x_stride < C || p->out_stride < C ||
        (p->residual && (p->residual_stride < C || p->residual_out_stride < C)))
        return DEP_ERR_INVALID_ARG;
    if (!aligned(p->x, 2) || !aligned(p->residual, 2) || !aligned(p->residual_out, 2) || !aligned(p->weight, 2) ||
        (!q8 && !aligned(p->out, 2)) || !aligned(p->scale, 4))
        return DEP_ERR_MISALIGNED;
    const int64_t ob = q8 ? 1 : 2;
    const Rows x{p->x, 2 * C, 2 * p->x_stride, R}, out{p->out, ob * C, ob * p->out_stride, R};
    const Rows w{p->weight, 2 * C, 2 * C, p->weight ? 1 : 0};
    const int64_t groups = p->quant == DEP_QUANT_INT8 ? 1 : (C + DEP_QUANT_GROUP - 1) / DEP_QUANT_GROUP;
    const Rows sc{p->scale, 4 * groups, 4 * groups, q8 ? R : 0};
    const Rows r{p->residual, 2 * C, 2 * p->residual_stride, p->residual ? R : 0};
    const Rows h{p->residual_out, 2 * C, 2 * p->residual_out_stride, p->residual ? R : 0};
    // Every block has read its row before it writes, so equal rows may be shared; anything else may not.
    if ((overlap(out, x) && !(p->out == p->x && !q8 && p->out_stride == p->x_stride)) || overlap(out, w) ||
        overlap(out, r) || overlap(out, h) || overlap(out, sc) || overlap(sc, x) || overlap(sc, w) ||
        overlap(sc, r) || overlap(sc, h) || overlap(h, w) ||
        (overlap(h, r) && !(p->residual_out == p->residual && p->residual_out_stride == p->residual_stride)) ||
        overlap(h, x))
        return DEP_ERR_INVALID_ARG;
    NormParams a{static_cast<const uint16_t *>(p->x),
                 static_cast<const uint16_t *>(p->residual),
                 static_cast<const uint16_t *>(p->weight),
                 static_cast<uint16_t *>(p->residual_out),
                 p->out,
                 p->scale,
                 p->x_stride,
                 p->residual_stride,
                 p->residual_out_stride,
                 p->out_stride,
                 R,
                 (int32_t)C,
                 p->eps};
    // Wide loads and stores where every row of every tensor allows them.
    const bool vec = C % 8 == 0 && x.aligned(16) && r.aligned(16) && h.aligned(16) && w.aligned(16) &&
                     out.aligned(q8 ? 8 : 16);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const cudaError_t e = vec ? norm_dispatch<true>(a, p->quant, norm, s) : norm_dispatch<false>(a, p->quant, norm, s);
    if (e != cudaSuccess) {
        cudaGetLastError();
        return DEP_ERR_CUDA;
    }
    return DEP_OK;
}

}  // namespace
}  // namespace dep

extern "C" {

dep_status_t dep_add_rms_norm(const dep_norm_args_t *args, void *stream)
{
    return dep::norm_entry(args, true, stream);
}

dep_status_t dep_quantize_rows(const dep_norm_args_t *args, void *stream)
{
    return dep::norm_entry(args, false, stream);
}

}  // extern "C"
