// delta_rule.cu -- the gated delta rule of a delta-attention layer.
//
//     S <- S diag(a),  S <- S + beta (v - S k) k^T,  o = scale S q,   a = exp(g)
//
// S [Dv, Dk] in FP32 for each (sequence, value head).  The rows of S (value
// channels) never meet: any set of rows can go to any warp.
//
// Recurrent kernel.  A group of eight lanes holds a row (Dk / 8 channels a lane,
// in chunks of four so that a group reads 128 consecutive bytes); a warp holds
// 4 * SETS rows.  The block turns a token's k, q and g into what all its rows need,
// once, through shared memory, and fetches the next token meanwhile.  The two dot
// products S k and S q are taken of the decayed state together, so each token costs one
// reduction: with u = beta (v - S k), o = scale (S q + u (k . q)) and S + u k^T.
// Bound: DRAM, the state read and written once (8 Dk Dv bytes a head): 64 sequences of 96
// heads of 128 x 128, 805 MB of states, 121 us (99 % of the copy rate); one sequence 4.1 us.
//
// Chunked kernel, for longer sequences: 16 tokens at a time as matrix products.
// With P_i = a_0 .. a_i, R_j = a_(j+1) .. a_15 and M_ij = a_(j+1) .. a_i (products of
// decays, channel by channel; never a quotient, so a decay of zero is as good as any),
//     A_ij = beta_i sum_c k_i k_j M_ij  (j < i),    B_ij = sum_c q_i k_j M_ij  (j <= i)
//     T = (I + A)^-1 diag(beta),   W = T (K.P),     U = T V - W S^T
//     O = (Q.P) S^T + B U,                          S <- S diag(P_15) + U^T (K.R)
// Two kernels.  delta_prepare_kernel works out what does not depend on the state (norms, decays, B,
// T, W, Q.P, K.R) for every chunk at once and leaves it in the workspace, as the operands of the
// state's MMAs; its four or five blocks an SM hide each other's latencies.  delta_state_kernel carries the
// states through the chunks: a warp holds 16 rows of S, as the accumulator of the last product, for
// the whole sequence: an accumulator fragment is also a left operand of the next product (with the
// channels in another order, the same on both sides), so S, U and the rest never leave the
// registers.  Two blocks of four warps an SM, 214 registers a thread (of 64 channels three, 168): with 128, sixteen warps an SM
// take longer (one sequence of 2048 tokens and 32 heads 403 us instead of 277, when both ran in 233),
// for want of loads under way; two warps for the two halves of the channels of 16 rows, whose sums
// have to meet in each chunk, 284 instead of 243.  Both kernels in one, preparing warps beside the
// state's, saved the way through memory (28 KB a chunk and head), but left SMs without work where
// sequences are few or of different lengths, and was never faster: that one sequence 498 us (now
// 235), 8192 tokens of 96 heads in 4 ragged sequences 1571 (now 1419), two sequences of 512 tokens
// and 76 heads, one for each SM, 151 (now 145).
// Precision: an FP32 operand is split into two parts of 11 bits, and three of the four products
// are kept (the last is below 2^-22): products of 22 bits instead of 24, sums and states in FP32.  On 8192 tokens the
// state is within 2.3e-7 of 64 bits (1.5e-7 if all is FP32).
// In the products with S and its update the parts are FP16, whose MMAs do twice TF32's work;
// what fits FP32's range is brought into FP16's by powers of two: one for each row of S and
// of U, from its largest value, and one for each token's k, q and W, from bounds on theirs.
// A and B are formed from TF32 parts, or, with one decay for all channels, from the BF16 tokens as
// they are (exact products, fewer of them and less memory, for five blocks an SM instead of four), T and W in FP32; V is BF16, and T meets it in three BF16
// parts.
// Measured: a chunk of one head takes 2.0 us of an SM to prepare (60 % of the issue slots), and 1.6
// in the state's kernel with one block on the SM, 2.5 for both of two.  Bound: the instructions of the
// one, the latencies of a chunk's chain in the other (the MMAs alone are 0.65 us a block).
// One scale for U and products with zeros above the diagonals join the tokens of a chunk: where that would show
// (infinities, NaN, tokens or states of far different size) the chunk's rows go token by token, see apart().
#include <cuda_bf16.h>

#include <algorithm>

#include "internal.h"
#include "layer.h"
#include "ptx.cuh"

namespace dep {
namespace {

struct DeltaParams {
    const uint16_t *q, *k, *v;
    const float *g, *beta;
    const float *s_in;
    float *s_out;
    uint16_t *o;
    const int32_t *cu, *slots;
    int64_t qs, ks, vs, gs, bs, os;
    int64_t tokens, n_states;
    int32_t n_seq, Hq, Hv, Dv;
    uint32_t flags;
    float scale;
    uint8_t *chunks;            // workspace
    int64_t chunk0, n_chunks;  // of this launch
};

constexpr uint32_t kEarly = 1u << 31;  // in flags: few chunks, see delta_prepare_kernel

__device__ __forceinline__ float lo_bf(uint32_t v) { return __uint_as_float(v << 16); }
__device__ __forceinline__ float hi_bf(uint32_t v) { return __uint_as_float(v & 0xFFFF0000u); }

// exp(g), at most one: the chunked kernel's scales count on decays that do not grow.
__device__ __forceinline__ float decay(float g) { return expf(g > 0.f ? 0.f : g); }

// First token and end of sequence s, clipped to the tensors.
__device__ __forceinline__ void seq_range(const DeltaParams &p, int s, int64_t &t0, int64_t &t1)
{
    if (p.cu) {
        const int64_t a = p.cu[s], b = p.cu[s + 1];
        t0 = a < 0 ? 0 : a > p.tokens ? p.tokens : a;
        t1 = b < t0 ? t0 : b > p.tokens ? p.tokens : b;
    } else {
        const int64_t len = p.tokens / p.n_seq;
        t0 = s * len;
        t1 = t0 + len;
    }
}

constexpr int kRecWarps = 4;

// Block: four warps, each 4 * SETS rows of one head of one sequence.
template <int DK, int SETS>
__global__ void __launch_bounds__(kRecWarps * 32) delta_recurrent_kernel(const DeltaParams p)
{
    constexpr int NV = DK / 32;  // float4 chunks a lane holds of a row
    __shared__ struct {
        float4 k[DK / 4], q[DK / 4], a[DK / 4];
        float kk[kRecWarps], qq[kRecWarps], kq[kRecWarps];
    } sm[2];  // the token's rows and their products, by turns
    const int slices = (p.Dv + kRecWarps * 4 * SETS - 1) / (kRecWarps * 4 * SETS);
    const int slice = blockIdx.x % slices, sh = blockIdx.x / slices;
    const int h = sh % p.Hv, s = sh / p.Hv;
    const int t = threadIdx.x, warp = t >> 5, lane = t & 31, l8 = lane & 7;
    const int row0 = (slice * kRecWarps + warp) * 4 * SETS + (lane >> 3);  // the lane's first row; the next are 4 on
    int64_t t0, t1;
    seq_range(p, s, t0, t1);
    const int64_t slot = p.slots ? p.slots[s] : s;
    if (slot < 0 || slot >= p.n_states) {  // padding: zeros out, no state
        for (int64_t tok = t0; tok < t1; ++tok)
#pragma unroll
            for (int i = 0; i < SETS; ++i)
                if (l8 == 0 && row0 + 4 * i < p.Dv)
                    p.o[tok * p.os + (int64_t)h * p.Dv + row0 + 4 * i] = 0;
        return;
    }
    const int64_t sbase = (slot * p.Hv + h) * (int64_t)p.Dv * DK;
    float4 S[SETS][NV];
#pragma unroll
    for (int i = 0; i < SETS; ++i)
#pragma unroll
        for (int c = 0; c < NV; ++c)
            S[i][c] = p.s_in && row0 + 4 * i < p.Dv
                          ? __ldcs(reinterpret_cast<const float4 *>(p.s_in + sbase + (int64_t)(row0 + 4 * i) * DK + 32 * c +
                                                                    4 * l8))
                          : make_float4(0.f, 0.f, 0.f, 0.f);
    const int hq = h / (p.Hv / p.Hq);
    const bool chan = (p.flags & DEP_DELTA_CHANNEL) != 0;
    // thread = channel for what a token brings; the lane's rows of v
    float k = 0.f, q = 0.f, g = 0.f, beta = 0.f, v[SETS];
    auto fetch = [&](int64_t tok) {
        if (t < DK) {
            k = __uint_as_float((uint32_t)p.k[tok * p.ks + (int64_t)hq * DK + t] << 16);
            q = __uint_as_float((uint32_t)p.q[tok * p.qs + (int64_t)hq * DK + t] << 16);
            g = p.g[tok * p.gs + (chan ? (int64_t)h * DK + t : h)];
        }
        beta = p.beta[tok * p.bs + h];
#pragma unroll
        for (int i = 0; i < SETS; ++i)
            v[i] = row0 + 4 * i < p.Dv
                       ? __uint_as_float((uint32_t)p.v[tok * p.vs + (int64_t)h * p.Dv + row0 + 4 * i] << 16)
                       : 0.f;
    };
    if (t0 < t1)
        fetch(t0);
    for (int64_t tok = t0; tok < t1; ++tok) {
        auto &m = sm[(tok - t0) & 1];
        if (t < DK) {
            reinterpret_cast<float *>(m.k)[t] = k;
            reinterpret_cast<float *>(m.q)[t] = q;
            reinterpret_cast<float *>(m.a)[t] = decay(g);
        }
        float kk = k * k, qq = q * q, kq = k * q;
#pragma unroll
        for (int d = 16; d; d >>= 1) {
            kk += __shfl_xor_sync(~0u, kk, d);
            qq += __shfl_xor_sync(~0u, qq, d);
            kq += __shfl_xor_sync(~0u, kq, d);
        }
        if (lane == 0) {
            m.kk[warp] = kk;
            m.qq[warp] = qq;
            m.kq[warp] = kq;
        }
        const float bt = beta;
        float vt[SETS];
#pragma unroll
        for (int i = 0; i < SETS; ++i)
            vt[i] = v[i];
        if (tok + 1 < t1)
            fetch(tok + 1);
        __syncthreads();
        kk = (m.kk[0] + m.kk[1]) + (m.kk[2] + m.kk[3]);
        qq = (m.qq[0] + m.qq[1]) + (m.qq[2] + m.qq[3]);
        kq = (m.kq[0] + m.kq[1]) + (m.kq[2] + m.kq[3]);
        float rq = p.scale, rk = 1.f;
        if (p.flags & DEP_DELTA_L2NORM) {
            rk = 1.0f / sqrtf(kk + 1e-6f);
            rq *= 1.0f / sqrtf(qq + 1e-6f);
        }
        kq *= rk * rq;
        float dk[SETS] = {}, dq[SETS] = {};
#pragma unroll
        for (int c = 0; c < NV; ++c) {
            const float4 kc = m.k[8 * c + l8], qc = m.q[8 * c + l8], ac = m.a[8 * c + l8];
#pragma unroll
            for (int i = 0; i < SETS; ++i) {
                float *sp = &S[i][c].x;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    sp[j] *= (&ac.x)[j];
                    dk[i] = fmaf(sp[j], (&kc.x)[j], dk[i]);
                    dq[i] = fmaf(sp[j], (&qc.x)[j], dq[i]);
                }
            }
        }
#pragma unroll
        for (int d = 4; d; d >>= 1)
#pragma unroll
            for (int i = 0; i < SETS; ++i) {
                dk[i] += __shfl_xor_sync(~0u, dk[i], d);
                dq[i] += __shfl_xor_sync(~0u, dq[i], d);
            }
#pragma unroll
        for (int i = 0; i < SETS; ++i) {
            const float u = bt * (vt[i] - dk[i] * rk);
            if (l8 == 0 && row0 + 4 * i < p.Dv)
                p.o[tok * p.os + (int64_t)h * p.Dv + row0 + 4 * i] =
                    __bfloat16_as_ushort(__float2bfloat16_rn(fmaf(u, kq, dq[i] * rq)));
            dk[i] = u * rk;
        }
#pragma unroll
        for (int c = 0; c < NV; ++c) {
            const float4 kc = m.k[8 * c + l8];
#pragma unroll
            for (int i = 0; i < SETS; ++i) {
                float *sp = &S[i][c].x;
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    sp[j] = fmaf(dk[i], (&kc.x)[j], sp[j]);
            }
        }
    }
#pragma unroll
    for (int i = 0; i < SETS; ++i)
#pragma unroll
        for (int c = 0; c < NV; ++c)
            if (row0 + 4 * i < p.Dv)
                __stcs(reinterpret_cast<float4 *>(p.s_out + sbase + (int64_t)(row0 + 4 * i) * DK + 32 * c + 4 * l8), S[i][c]);
}

template <int DK, int SETS>
cudaError_t recurrent_launch(const DeltaParams &p, cudaStream_t s)
{
    const int64_t slices = (p.Dv + kRecWarps * 4 * SETS - 1) / (kRecWarps * 4 * SETS);
    const int64_t blocks = slices * p.Hv * p.n_seq;
    if (blocks > INT32_MAX)
        return cudaErrorInvalidConfiguration;
    delta_recurrent_kernel<DK, SETS><<<(unsigned)blocks, kRecWarps * 32, 0, s>>>(p);
    return cudaGetLastError();
}

// ---------------------------------------------------------------------------------
// chunked kernel

constexpr int kC = 16;            // tokens of a chunk
constexpr int kPrep = 128;        // threads that prepare a chunk
constexpr int kStateWarps = 4;    // of a block, 16 rows of the state each
constexpr int kRows = 16 * kStateWarps;
constexpr int kStages = 2;        // chunks in a block's ring
constexpr int kTT = 20;           // row stride of 16-wide matrices in shared memory

// v = hi + lo, hi rounded to TF32's 11 bits (half away from zero) by integer arithmetic: the
// conversion instruction runs at an eighth of its rate.  The MMA ignores what lo has below 11 bits.
// A NaN may leave hi, but not lo.
__device__ __forceinline__ void tf32_split(float v, uint32_t &hi, uint32_t &lo)
{
    hi = (__float_as_uint(v) + 0x1000u) & 0xFFFFE000u;
    lo = __float_as_uint(v - __uint_as_float(hi));
}
__device__ __forceinline__ void mma_tf32(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1)
{
    asm("mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// The accumulator fragment c as a left operand: its columns 2t and 2t + 1 become k = t and t + 4.
__device__ __forceinline__ void split_a(const float (&c)[4], uint32_t (&hi)[4], uint32_t (&lo)[4])
{
    tf32_split(c[0], hi[0], lo[0]);
    tf32_split(c[2], hi[1], lo[1]);
    tf32_split(c[1], hi[2], lo[2]);
    tf32_split(c[3], hi[3], lo[3]);
}
__device__ __forceinline__ void mma_f16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1)
{
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// Two values (low half first) as FP16, and what that leaves of them.
__device__ __forceinline__ void f16_split2(float a, float b, uint32_t &hi, uint32_t &lo)
{
    const __half2 h = __floats2half2_rn(a, b);
    const float2 f = __half22float2(h);
    const __half2 l = __floats2half2_rn(a - f.x, b - f.y);
    hi = *reinterpret_cast<const uint32_t *>(&h);
    lo = *reinterpret_cast<const uint32_t *>(&l);
}
// N products d[n] += a b[n] of FP16 parts, each as three: the small ones first, and those of one d
// N MMAs apart (an MMA takes 24 cycles, a warp issues one in 8).
template <int N>
__device__ __forceinline__ void mma_f16x3(float (*const (&d)[N])[4], const uint32_t (&ah)[4], const uint32_t (&al)[4],
                                          const uint4 (&b)[N])
{
#pragma unroll
    for (int n = 0; n < N; ++n)
        mma_f16(*d[n], al, b[n].x, b[n].y);
#pragma unroll
    for (int n = 0; n < N; ++n)
        mma_f16(*d[n], ah, b[n].z, b[n].w);
#pragma unroll
    for (int n = 0; n < N; ++n)
        mma_f16(*d[n], ah, b[n].x, b[n].y);
}
__device__ __forceinline__ void mma_bf16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1)
{
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// Three BF16 parts of two values: all of FP32's 24 bits.
__device__ __forceinline__ void bf16_split3(float a, float b, uint32_t &p0, uint32_t &p1, uint32_t &p2)
{
    const auto part = [](float &x, float &y) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(x, y);
        const uint32_t w = *reinterpret_cast<const uint32_t *>(&h);
        x -= lo_bf(w);
        y -= hi_bf(w);
        return w;
    };
    p0 = part(a, b);
    p1 = part(a, b);
    p2 = part(a, b);
}
// The power of two that brings values of up to `top` below 2^14 (top's exponent to 13), and its
// reciprocal.  Tops below 2^-107 count as that.
__device__ __forceinline__ float scale_for(float top, float &inv)
{
    const int e = max((int)(__float_as_uint(top) >> 23), 20);
    inv = __uint_as_float((uint32_t)(e - 13) << 23);
    return __uint_as_float((uint32_t)(267 - e) << 23);
}
__device__ __forceinline__ float max3_abs(float a, float b, float c)
{
    float r;
    asm("max.abs.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}
__device__ __forceinline__ float row_max(float v)  // over the four lanes of a row
{
    v = fmaxf(v, __shfl_xor_sync(~0u, v, 1));
    return fmaxf(v, __shfl_xor_sync(~0u, v, 2));
}
__device__ __forceinline__ float2 ld2(const float *p) { return *reinterpret_cast<const float2 *>(p); }

constexpr float kUnB = 16.f;  // B is stored times the scales of q and k, which make it up to 2^16, over this
constexpr float kUnO = 0x1p24f;  // outputs are added up over this: before q's scale they may be 2^35 times the state
// Of a row of S.  Rows whose largest value is below 2^-92 have fewer bits left in the products; S itself is as FP32
// holds it.
constexpr float kMostScale = 0x1p100f;
constexpr int kSort = 256;

constexpr float kLeastQ = 0x1p-70f * kUnO;  // what undoes a q's scale is not less, but for a q of zeros (or below 2^-63)

// Least output (before q's scale) of a row whose U' has the scale 1 / j that does not have to be looked at: 16 in the units
// of U' B'.  None where the row's U is zero (or below 2^-107).
__device__ __forceinline__ float least_for(float j) { return j > 0x1p-120f ? j * (16.f * kUnB / kUnO) : 0.f; }

// The sequence of rank r by length, longest first: blocks start in order, and a long
// sequence that starts last leaves the other SMs idle.  Tables of more than kSort
// sequences are taken as they are.
__device__ __forceinline__ int longest_first(const DeltaParams &p, int r, int (&len)[kSort + 1])
{
    const int n = p.n_seq;
    if (!p.cu || n < 2 || n > kSort)
        return r;
    for (int t = threadIdx.x; t < n; t += 32 * kStateWarps) {
        int64_t t0, t1;
        seq_range(p, t, t0, t1);
        len[t] = (int)(t1 - t0);
    }
    __syncthreads();
    for (int t = threadIdx.x; t < n; t += 32 * kStateWarps) {
        int rank = 0;
        for (int j = 0; j < n; ++j)
            rank += len[j] > len[t] || (len[j] == len[t] && j < t);
        if (rank == r)
            len[kSort] = t;
    }
    __syncthreads();
    return len[kSort];
}

__device__ __forceinline__ void cp_async16(void *dst, const void *src, bool in)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"((uint32_t)__cvta_generic_to_shared(dst)), "l"(src),
                 "r"(in ? 16 : 0)
                 : "memory");
}

// What an MMA's lane (g, t) takes of a right operand, 16 bytes: FP16 parts of the k's 2t, 2t + 1
// (x) and 2t + 8, 2t + 9 (y) of its sixteen, and the parts that those leave (z, w).  Rows and lanes
// are laid out such that the eight lanes of a load phase meet no bank twice.
template <int DK>
struct Chunk {  // of one head: what its state needs of sixteen tokens
    uint4 qp[kC][DK / 4];  // Q.P by token, sixteen channels after another, four lanes t each, at ^ 4 in odd rows
    uint4 B[kC][4];        // B by row
    uint4 T01[kC][4];      // T by row, in BF16 parts: the first two,
    uint2 T2[kC][4];       // and the third
    float last[DK];        // P_15
    float iw[kC], ik[kC], iq[kC], unused[kC];  // what undoes the scales of W, k and q (and kUnO); to a multiple of 128 bytes
    uint4 kr[DK][4];       // K.R by channel; lane t at t ^ (channel / 2 % 4)
    uint4 w[kC][DK / 4];   // W, as Q.P
};

// Chunks are numbered through all sequences, from t0 / 16 + s on for sequence s: no two share a
// number, and there are tokens / 16 + n_seq at most.
__device__ __forceinline__ int64_t first_chunk(const DeltaParams &p, int s)
{
    int64_t t0, t1;
    seq_range(p, s, t0, t1);
    return t0 / kC + s;
}

template <int DK, bool CHAN>
struct PrepShared {
    static constexpr int KS = DK + 8;  // float2 reads without conflicts
    struct Level {                     // operands of the products of one level: rows k_i then q_i, columns k_j
        float row[16][KS], col[8][KS];
    };
    struct Raw {  // the tokens as they are; rows off by 16 bytes for ldmatrix
        uint16_t k[kC][DK + 8], q[kC][DK + 8];
        float g[CHAN ? kC : 1][DK];
    };
    // One after another in this memory: the tokens and the levels, where the chunk's K.R and W come to lie.
    static constexpr int HEAD = offsetof(Chunk<DK>, kr);
    static constexpr int BODY = CHAN ? 2 * (int)sizeof(Level) : (int)sizeof(Chunk<DK>) - HEAD;
    static_assert(sizeof(Raw) <= BODY && sizeof(Chunk<DK>) <= HEAD + BODY && HEAD % 16 == 0, "");
    alignas(128) uint8_t mem[HEAD + BODY];
    alignas(16) float A[kC][kC];
    alignas(16) float T[kC][kTT], Tk[kC][kTT];  // columns of T, and of T over k's scales
    alignas(16) float other[4][32][4];          // halves of the levels' products
    alignas(16) float pair[CHAN ? 1 : 4][2][kC][kC];  // each warp's part of k_i k_j, and of q_i k_j
    alignas(16) float part[4][48], norm[4][48], inv[4][32], sw[4][kC], beta[kC], g[kC];
};

// One block for each chunk and head.
// A and B come from matrix products, level by level.  At level b (1, 2, 4, 8) token i, whose
// bit b is set, is a row and meets the columns j that share its bits above b and have
// that bit clear: M_ij is the product of the decays from the row's group of b tokens
// on up to i, times that of the decays after j up to the group's end.  Every pair j < i
// meets at one level, the highest bit in which the two differ.  (With one decay for all channels
// M_ij is a number, and one product of all tokens with all will do.)
// A thread works on one channel; of 64 channels two threads each, one with what tokens need
// (Q.P, W), the other with what pairs need (the levels, K.R).
template <int DK, bool CHAN>
__global__ void __launch_bounds__(kPrep, CHAN ? 4 : 5) delta_prepare_kernel(const DeltaParams p)
{
    extern __shared__ __align__(128) uint8_t smem_raw[];
    auto &pr = *reinterpret_cast<PrepShared<DK, CHAN> *>(smem_raw);
    auto &sg = *reinterpret_cast<Chunk<DK> *>(pr.mem);
    auto &raw = *reinterpret_cast<typename PrepShared<DK, CHAN>::Raw *>(pr.mem + PrepShared<DK, CHAN>::HEAD);
    auto *level = reinterpret_cast<typename PrepShared<DK, CHAN>::Level *>(pr.mem + PrepShared<DK, CHAN>::HEAD);
    // The state's kernel may start at once if these blocks are few, two for an SM; else when all are done: while
    // others still work its first blocks would meet on the few SMs that are free (one sequence of 4096 tokens and
    // 32 heads: 522 us at once, 472 late; 16 tokens of 32 heads: 9.2 and 10.8).
    const bool early = (p.flags & kEarly) != 0;
    if (early)
        griddep_launch_dependents();
    const int h = blockIdx.x % p.Hv, pt = threadIdx.x, pw = pt >> 5, lane = pt & 31;
    const int64_t local = blockIdx.x / p.Hv, number = p.chunk0 + local;
    int s = 0;
    for (int n = p.n_seq; n > 1;) {  // the last sequence that starts at or before this chunk
        const int step = (n + 31) / 32;
        const bool before = lane * step < n && first_chunk(p, s + lane * step) <= number;
        const int at = max(31 - __clz(__ballot_sync(~0u, before)), 0) * step;
        s += at;
        n = min(step, n - at);
    }
    int64_t t0, t1;
    seq_range(p, s, t0, t1);
    const int64_t len = t1 - t0, first = (number - t0 / kC - s) * kC;  // of its tokens
    if (first < 0 || first >= len)
        return;
    const int left = (int)(len - first < kC ? len - first : kC);
    const bool l2 = (p.flags & DEP_DELTA_L2NORM) != 0;
    const int ch = pt % DK;
    const bool tokens = pt < DK, pairs = pt >= kPrep - DK;
    const int hq = h / (p.Hv / p.Hq);
    const uint16_t *k0 = p.k + t0 * p.ks + (int64_t)hq * DK, *q0 = p.q + t0 * p.qs + (int64_t)hq * DK;
    const float *gp = p.g + t0 * p.gs + (CHAN ? (int64_t)h * DK : h);
    {
        constexpr int QC = DK / 8, GC = DK / 4;  // 16-byte pieces of a token
#pragma unroll
        for (int i = pt; i < kC * QC; i += kPrep) {
            const int tok = i / QC, e = i % QC * 8;
            const int64_t at = first + (tok < left ? tok : 0);
            cp_async16(&raw.k[tok][e], k0 + at * p.ks + e, tok < left);
            cp_async16(&raw.q[tok][e], q0 + at * p.qs + e, tok < left);
        }
        if (CHAN)
#pragma unroll
            for (int i = pt; i < kC * GC; i += kPrep) {
                const int tok = i / GC, e = i % GC * 4;
                cp_async16(&raw.g[tok][e], gp + (first + (tok < left ? tok : 0)) * p.gs + e, tok < left);
            }
        asm volatile("cp.async.commit_group;" ::: "memory");
        if (pt < kC) {
            pr.beta[pt] = pt < left ? p.beta[(t0 + first + pt) * p.bs + h] : 0.f;
            pr.g[pt] = !CHAN && pt < left ? decay(gp[(first + pt) * p.gs]) : 1.f;
        }
    }
    for (int i = pt; i < kC * 4; i += kPrep)  // above the diagonal B stays zero
        (&sg.B[0][0])[i] = make_uint4(0, 0, 0, 0);
    for (int i = pt; i < kC * kC; i += kPrep)
        (&pr.A[0][0])[i] = 0.f;
    auto put_b = [&](int i, int j, float v) {  // B_ij into its lane's sixteen bytes
        uint32_t hi, lo;
        f16_split2(v * (1.f / kUnB), 0.f, hi, lo);
        uint16_t *d = reinterpret_cast<uint16_t *>(&sg.B[i][(j & 7) >> 1]) + (j >> 3) * 2 + (j & 1);
        d[0] = (uint16_t)hi;
        d[4] = (uint16_t)lo;
    };
    // this channel's place in a row of W or Q.P, in FP16 numbers: its lane's sixteen bytes
    const int c16 = ch & 15, at = ((ch >> 4) * 4 + ((c16 & 7) >> 1)) * 8 + (c16 >> 3) * 2 + (c16 & 1);
    asm volatile("cp.async.wait_group 0;" ::: "memory");
    __syncthreads();
    float k[kC], q[kC], a[kC], kp[kC];  // kp: K.P
#pragma unroll
    for (int i = 0; i < kC; ++i) {
        k[i] = __uint_as_float((uint32_t)raw.k[i][ch] << 16);
        q[i] = __uint_as_float((uint32_t)raw.q[i][ch] << 16);
        a[i] = CHAN ? decay(raw.g[i][ch]) : pr.g[i];
    }
    {
        // Each token's sums of k k, q q and k q over the channels: the diagonals of products of the BF16
        // rows with themselves, warp pw a quarter of the channels.  A left operand's registers hold the
        // right operands of its two halves, too.
        constexpr int KW = DK / 64;  // steps of 16 channels
        float kk[2][4] = {}, qq[2][4] = {}, qk[2][4] = {};
#pragma unroll
        for (int i = 0; i < KW; ++i) {
            const int col = (pw * KW + i) * 16 + 8 * (lane >> 4), row = lane & 15;
            uint32_t x[4], y[4];
            asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                         : "=r"(x[0]), "=r"(x[1]), "=r"(x[2]), "=r"(x[3])
                         : "r"((uint32_t)__cvta_generic_to_shared(&raw.k[row][col]))
                         : "memory");
            asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                         : "=r"(y[0]), "=r"(y[1]), "=r"(y[2]), "=r"(y[3])
                         : "r"((uint32_t)__cvta_generic_to_shared(&raw.q[row][col]))
                         : "memory");
#pragma unroll
            for (int n = 0; n < 2; ++n) {
                mma_bf16(kk[n], x, x[n], x[2 + n]);
                mma_bf16(qq[n], y, y[n], y[2 + n]);
                mma_bf16(qk[n], y, x[n], x[2 + n]);
            }
        }
        const int g = lane >> 2;
        if ((lane & 3) == g >> 1) {  // this lane holds the diagonal at g and g + 8
#pragma unroll
            for (int n = 0; n < 2; ++n) {
                pr.part[pw][8 * n + g] = g & 1 ? kk[n][2 * n + 1] : kk[n][2 * n];
                pr.part[pw][16 + 8 * n + g] = g & 1 ? qq[n][2 * n + 1] : qq[n][2 * n];
                pr.part[pw][32 + 8 * n + g] = g & 1 ? qk[n][2 * n + 1] : qk[n][2 * n];
            }
        }
        if (!CHAN)  // all pairs
#pragma unroll
            for (int n = 0; n < 2; ++n)
#pragma unroll
                for (int e = 0; e < 4; e += 2) {
                    const int i = g + 4 * e, j = 8 * n + 2 * (lane & 3);
                    *reinterpret_cast<float2 *>(&pr.pair[pw][0][i][j]) = make_float2(kk[n][e], kk[n][e + 1]);
                    *reinterpret_cast<float2 *>(&pr.pair[pw][1][i][j]) = make_float2(qk[n][e], qk[n][e + 1]);
                }
        __syncthreads();
        // every warp finishes the sums for itself
        const float sum = (pr.part[0][lane] + pr.part[1][lane]) + (pr.part[2][lane] + pr.part[3][lane]);
        const float f = (lane < 16 ? 1.f : p.scale) * (l2 ? 1.f / sqrtf(sum + 1e-6f) : 1.f);
        // 2^e > the norm of the normalised row >= its largest value; rows are taken times 2^(8 - e) from here on
        const int e = (((int)(__float_as_uint(sum * f * f) >> 23) - 127 + 2) >> 1);
        pr.norm[pw][lane] = f * __uint_as_float((uint32_t)(127 + 8 - e) << 23);
        pr.inv[pw][lane] = __uint_as_float((uint32_t)(127 - 8 + e) << 23);
        if (lane < 16)
            pr.norm[pw][32 + lane] = (pr.part[0][32 + lane] + pr.part[1][32 + lane]) +
                                     (pr.part[2][32 + lane] + pr.part[3][32 + lane]);
        __syncwarp();
    }
    if (pt < kC)
        put_b(pt, pt, pr.norm[pw][32 + pt] * pr.norm[pw][pt] * pr.norm[pw][16 + pt]);
    if (pt < 32)
        (pt < 16 ? sg.ik : sg.iq)[pt & 15] = pr.inv[pw][pt] * (pt < 16 ? 1.f : kUnO);
#pragma unroll
    for (int i = 0; i < kC; i += 4) {
        const float4 nk = *reinterpret_cast<const float4 *>(&pr.norm[pw][i]);
        const float4 nq = *reinterpret_cast<const float4 *>(&pr.norm[pw][16 + i]);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            k[i + e] *= (&nk.x)[e];
            q[i + e] *= (&nq.x)[e];
        }
    }
    if (tokens) {
        float P = 1.f;
#pragma unroll
        for (int i = 0; i < kC; i += 2) {
            const float P0 = P * a[i], P1 = P0 * a[i + 1];
            P = P1;
            kp[i] = k[i] * P0;
            kp[i + 1] = k[i + 1] * P1;
            uint32_t hi, lo;
            f16_split2(q[i] * P0, q[i + 1] * P1, hi, lo);
            uint16_t *d0 = reinterpret_cast<uint16_t *>(&sg.qp[i][0]) + at;
            uint16_t *d1 = reinterpret_cast<uint16_t *>(&sg.qp[i + 1][0]) + (at ^ 32);
            d0[0] = (uint16_t)hi;
            d0[4] = (uint16_t)lo;
            d1[0] = (uint16_t)(hi >> 16);
            d1[4] = (uint16_t)(lo >> 16);
        }
        sg.last[ch] = P;
    }
    if (CHAN) {
        float mine[4];  // of this warp's level
#pragma unroll
        for (int l0 = 0; l0 < 4; l0 += 2) {  // two levels at a time, half of the channels for each warp
            if (pairs)
#pragma unroll
                for (int l = l0; l < l0 + 2; ++l) {
                    const int b = 1 << l;
                    float f = 1.f;
#pragma unroll
                    for (int r = 0; r < 8; ++r) {
                        const int i = (r & ~(b - 1)) << 1 | b | (r & (b - 1));
                        f = i % b == 0 ? a[i] : f * a[i];
                        level[l & 1].row[r][ch] = k[i] * f;
                        level[l & 1].row[8 + r][ch] = q[i] * f;
                    }
#pragma unroll
                    for (int n = 7; n >= 0; --n) {
                        const int j = (n & ~(b - 1)) << 1 | (n & (b - 1));
                        f = j % b == b - 1 ? 1.f : f * a[j + 1];
                        level[l & 1].col[n][ch] = k[j] * f;
                    }
                }
            __syncthreads();
            const int g = lane >> 2, t = lane & 3;
            const auto &lv = level[pw & 1];
            float d[3][4] = {};  // one for each of the three products
#pragma unroll
            for (int i = 0; i < DK / 16; ++i) {
                const int at = 8 * (pw / 2 * (DK / 16) + i) + 2 * t;
                const float2 lo = ld2(&lv.row[g][at]), hi = ld2(&lv.row[g + 8][at]), cb = ld2(&lv.col[g][at]);
                const float c4[4] = {lo.x, lo.y, hi.x, hi.y};
                uint32_t ah[4], al[4];
                split_a(c4, ah, al);
                uint32_t h0, l0, h1, l1;
                tf32_split(cb.x, h0, l0);
                tf32_split(cb.y, h1, l1);
                mma_tf32(d[2], al, h0, h1);
                mma_tf32(d[1], ah, l0, l1);
                mma_tf32(d[0], ah, h0, h1);
            }
            // one of the two warps of a level finishes it: of the first two levels 2 and 3, of the others 0 and 1
#pragma unroll
            for (int e = 0; e < 4; ++e)
                d[0][e] += d[2][e] + d[1][e];
            if ((l0 == 0) == (pw >= 2))
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    mine[e] = d[0][e];
            else
                *reinterpret_cast<float4 *>(pr.other[pw ^ 2][lane]) = make_float4(d[0][0], d[0][1], d[0][2], d[0][3]);
            __syncthreads();
        }
        {
            const int g = lane >> 2, t = lane & 3, b = 1 << (pw ^ 2);
            const float4 other = *reinterpret_cast<const float4 *>(pr.other[pw][lane]);
            const int i = (g & ~(b - 1)) << 1 | b | (g & (b - 1));
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int n = 2 * t + e, j = (n & ~(b - 1)) << 1 | (n & (b - 1));
                if ((n & ~(b - 1)) == (g & ~(b - 1))) {
                    pr.A[i][j] = (mine[e] + (&other.x)[e]) * (pr.inv[pw][i] * pr.inv[pw][j]);
                    put_b(i, j, mine[2 + e] + (&other.x)[2 + e]);
                }
            }
        }
    } else {
        // One decay for all channels: M is a number, and the pairs' products are those of the tokens as they are.
        const int i = pt >> 3, j0 = 2 * (pt & 7);
        float2 kk2 = make_float2(0.f, 0.f), qk2 = kk2;
#pragma unroll
        for (int w = 0; w < 4; ++w) {
            const float2 a = ld2(&pr.pair[w][0][i][j0]), b = ld2(&pr.pair[w][1][i][j0]);
            kk2.x += a.x, kk2.y += a.y;
            qk2.x += b.x, qk2.y += b.y;
        }
#pragma unroll
        for (int j = j0; j < j0 + 2; ++j) {
            const float kk = j == j0 ? kk2.x : kk2.y, qk = j == j0 ? qk2.x : qk2.y;
            float M = 1.f;
#pragma unroll
            for (int m = 1; m < kC; ++m)
                M *= m > j && m <= i ? pr.g[m] : 1.f;
            if (j < i) {
                pr.A[i][j] = kk * M * ((pr.norm[pw][i] * pr.inv[pw][i]) * (pr.norm[pw][j] * pr.inv[pw][j]));
                put_b(i, j, qk * M * pr.norm[pw][16 + i] * pr.norm[pw][j]);  // (the norms of zeros have no finite product)
            }
        }
    }
    __syncthreads();
    if (pairs) {
        float R = 1.f;
#pragma unroll
        for (int i = kC - 1; i >= 0; --i) {
            k[i] *= R;
            R *= a[i];
        }
    }
    if (pairs)
#pragma unroll
        for (int t = 0; t < 4; ++t) {
            uint4 v;
            f16_split2(k[2 * t], k[2 * t + 1], v.x, v.z);
            f16_split2(k[2 * t + 8], k[2 * t + 9], v.y, v.w);
            sg.kr[ch][t ^ (ch >> 1 & 3)] = v;
        }
    if (pw == 0) {  // T: lane j solves (I + A) x = e_j, then times beta_j
        const int j = lane & 15;
        float x[kC];
#pragma unroll
        for (int i = 0; i < kC; ++i) {
            float d0 = 0.f, d1 = 0.f;
#pragma unroll
            for (int m = 0; m < i; m += 4) {
                const float4 r = *reinterpret_cast<const float4 *>(&pr.A[i][m]);
#pragma unroll
                for (int e = 0; e < 4 && m + e < i; ++e)
                    (e & 1 ? d1 : d0) = fmaf((&r.x)[e], x[m + e], e & 1 ? d1 : d0);
            }
            x[i] = (i == j ? 1.f : 0.f) - pr.beta[i] * (d0 + d1);
        }
        const float b = pr.beta[j], bk = b * pr.inv[pw][j];
        if (lane < 16)
#pragma unroll
            for (int i = 0; i < kC; i += 4) {  // x is zero above its own row
                *reinterpret_cast<float4 *>(&pr.T[j][i]) = make_float4(x[i] * b, x[i + 1] * b, x[i + 2] * b, x[i + 3] * b);
                *reinterpret_cast<float4 *>(&pr.Tk[j][i]) =
                    make_float4(x[i] * bk, x[i + 1] * bk, x[i + 2] * bk, x[i + 3] * bk);
            }
    }
    __syncthreads();
    if (pt < 4 * kC) {  // T for the state's warps
        const int i = pt >> 2, t = pt & 3;
        uint4 p01;
        uint2 p2;
        bf16_split3(pr.T[2 * t][i], pr.T[2 * t + 1][i], p01.x, p01.z, p2.x);
        bf16_split3(pr.T[2 * t + 8][i], pr.T[2 * t + 9][i], p01.y, p01.w, p2.y);
        sg.T01[i][t] = p01;
        sg.T2[i][t] = p2;
    }
    if (tokens) {
        // |W_i| <= sum_j |T_ij| times the bound on k_j's values, 2^8 over its scale
        float top = 0.f, inv;
        if (lane < kC)
#pragma unroll
            for (int j = 0; j < kC; ++j)
                top += fabsf(pr.Tk[j][lane]);
        const float s = scale_for(256.f * top, inv);
        if (lane < kC)
            pr.sw[pw][lane] = s;
        if (pw == 0 && lane < kC)
            sg.iw[lane] = inv;
        float w[kC] = {};
#pragma unroll
        for (int j = 0; j < kC; ++j)
#pragma unroll
            for (int i = j & ~3; i < kC; i += 4) {
                const float4 c4 = *reinterpret_cast<const float4 *>(&pr.Tk[j][i]);
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    w[i + e] = fmaf((&c4.x)[e], kp[j], w[i + e]);
            }
        __syncwarp();
#pragma unroll
        for (int i = 0; i < kC; i += 2) {
            const float2 s2 = ld2(&pr.sw[pw][i]);
            uint32_t hi, lo;
            f16_split2(w[i] * s2.x, w[i + 1] * s2.y, hi, lo);
            uint16_t *d0 = reinterpret_cast<uint16_t *>(&sg.w[i][0]) + at;
            uint16_t *d1 = reinterpret_cast<uint16_t *>(&sg.w[i + 1][0]) + (at ^ 32);
            d0[0] = (uint16_t)hi;
            d0[4] = (uint16_t)lo;
            d1[0] = (uint16_t)(hi >> 16);
            d1[4] = (uint16_t)(lo >> 16);
        }
    }
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    __syncthreads();
    if (!early)
        griddep_launch_dependents();
    if (pt == 0) {
        asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(
                         p.chunks + (local * p.Hv + h) * (int64_t)sizeof(Chunk<DK>)),
                     "r"((uint32_t)__cvta_generic_to_shared(pr.mem)), "r"((int)sizeof(Chunk<DK>))
                     : "memory");
        asm volatile("cp.async.bulk.commit_group;" ::: "memory");
        asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
    }
}

template <int DK>
struct StateShared {
    Chunk<DK> stage[kStages];
    uint16_t v[kStateWarps][kC][24];  // each warp's part of V, then of O; rows off a multiple of 128 bytes
    int order[kSort + 1];
    int head;
    int64_t token, end;  // first of this launch's, and the sequence's end
};

// One block for each sequence, head and kRows rows of its state.
template <int DK>
__global__ void __launch_bounds__(32 * kStateWarps, DK == 64 ? 3 : 2) delta_state_kernel(const DeltaParams p)
{
    extern __shared__ __align__(128) uint8_t smem_raw[];
    auto &sm = *reinterpret_cast<StateShared<DK> *>(smem_raw);
    const int slices = (p.Dv + kRows - 1) / kRows;
    const int slice = blockIdx.x % slices, sh = blockIdx.x / slices;
    const int h = sh % p.Hv, s = longest_first(p, sh / p.Hv, sm.order);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    int64_t t0, t1;
    seq_range(p, s, t0, t1);
    const int64_t slot = p.slots ? p.slots[s] : s;
    const int64_t len = t1 - t0, all = (len + kC - 1) / kC, base = t0 / kC + s - p.chunk0;
    if (slot < 0 || slot >= p.n_states) {  // padding: zeros out, no state
        griddep_wait();
        const int rows = p.Dv - slice * kRows < kRows ? p.Dv - slice * kRows : kRows;
        if (p.chunk0 == 0)
            for (int64_t i = threadIdx.x; i < len * rows; i += blockDim.x)
                p.o[(t0 + i / rows) * p.os + (int64_t)h * p.Dv + slice * kRows + i % rows] = 0;
        return;
    }
    // chunks from .. to of the sequence are among those of this launch
    const int64_t from = base < 0 ? -base : 0, to = all < p.n_chunks - base ? all : p.n_chunks - base;
    if (from >= to && !(all == 0 && base >= 0 && base < p.n_chunks)) {
        griddep_wait();  // no block ends before the chunks are done: what follows this kernel counts on both
        return;
    }
    const int64_t chunks = to - from;
    const float *s_in = from > 0 ? p.s_out : p.s_in;
    const int64_t sbase = (slot * p.Hv + h) * (int64_t)p.Dv * DK;
    const uint8_t *src = p.chunks + ((base + from) * p.Hv + h) * (int64_t)sizeof(Chunk<DK>);
    constexpr int kPieces = ((int)sizeof(Chunk<DK>) / 16 + 32 * kStateWarps - 1) / (32 * kStateWarps);
    // Pieces i0 .. i0 + n - 1 that this thread copies of chunk c.
    auto fetch = [&](int64_t c, int i0, int n) {
        const uint8_t *at = src + c * p.Hv * (int64_t)sizeof(Chunk<DK>) + 16 * threadIdx.x;
        const uint32_t to = (uint32_t)__cvta_generic_to_shared(&sm.stage[c % kStages]) + 16 * threadIdx.x;
#pragma unroll
        for (int i = i0; i < i0 + n; ++i)
            if (c < chunks && i < kPieces &&
                (16 * 32 * kStateWarps * (i + 1) <= (int)sizeof(Chunk<DK>) ||
                 16 * (32 * kStateWarps * i + (int)threadIdx.x) < (int)sizeof(Chunk<DK>)))
                asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to + 16 * 32 * kStateWarps * i),
                             "l"(at + 16 * 32 * kStateWarps * i));
    };
    auto commit = [] { asm volatile("cp.async.commit_group;" ::: "memory"); };
    auto &mine = sm.v[warp];
    auto fetch_v = [&](int64_t c) {
        const int64_t tok = (from + c) * kC + (lane >> 1);
        const int row = (slice * kStateWarps + warp) * 16 + 8 * (lane & 1);
        return c < chunks && tok < len && row < p.Dv
                   ? *reinterpret_cast<const uint4 *>(p.v + (t0 + tok) * p.vs + (int64_t)h * p.Dv + row)
                   : make_uint4(0, 0, 0, 0);
    };
    uint4 v = fetch_v(0);
    const int row0 = (slice * kStateWarps + warp) * 16, g = lane >> 2, t = lane & 3;
    const bool live = row0 < p.Dv;  // Dv is a multiple of 16
    constexpr int NT = DK / 8;
    float S[NT][4];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        float2 a = make_float2(0.f, 0.f), b = a;
        if (live && s_in) {
            a = *reinterpret_cast<const float2 *>(s_in + sbase + (int64_t)(row0 + g) * DK + 8 * n + 2 * t);
            b = *reinterpret_cast<const float2 *>(s_in + sbase + (int64_t)(row0 + g + 8) * DK + 8 * n + 2 * t);
        }
        S[n][0] = a.x;
        S[n][1] = a.y;
        S[n][2] = b.x;
        S[n][3] = b.y;
    }
    // S is held times a power of two for each row: r0 for row g, r1 for row g + 8, such that the row's largest
    // value lies in [2^8, 2^15), or the scale at its limit.
    float r0 = 1.f, r1 = 1.f, i0 = 1.f, i1 = 1.f;  // the scales, and what undoes them
    auto rescale = [&](float f0, float f1) {
#pragma unroll
        for (int n = 0; n < NT; ++n)
            S[n][0] *= f0, S[n][1] *= f0, S[n][2] *= f1, S[n][3] *= f1;
        r0 *= f0, r1 *= f1;
        i0 = 1.f / r0, i1 = 1.f / r1;
    };
    auto factor = [](float top, float r) {  // what brings a row back into its range
        float inv;
        return top >= 32768.f || (top < 256.f && top > 0.f && r < kMostScale)
                   ? fminf(scale_for(top, inv), kMostScale / r)
                   : 1.f;
    };
    auto keep_range = [&](float m0, float m1) {  // the lane's largest values of both rows
        // Mostly every row has a value of 2^8 or more, and none of 2^15: one bit in each row's four of `some`.
        unsigned some = __ballot_sync(~0u, m0 >= 256.f), some1 = __ballot_sync(~0u, m1 >= 256.f);
        some |= some >> 1, some1 |= some1 >> 1;
        some = (some | some >> 2) & (some1 | some1 >> 2) & 0x11111111u;
        if (__any_sync(~0u, !(fmaxf(m0, m1) < 32768.f)) || some != 0x11111111u)
            rescale(factor(row_max(m0), r0), factor(row_max(m1), r1));
    };
    auto start_range = [&] {
        float m0 = 0.f, m1 = 0.f;
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            m0 = max3_abs(m0, S[n][0], S[n][1]);
            m1 = max3_abs(m1, S[n][2], S[n][3]);
        }
        keep_range(m0, m1);
    };
    start_range();
    // Whether a chunk's tokens are too far apart for one product.  U' has one scale for each row, set by its largest
    // token, and what is below 2^-25 in its units is lost.  So an output has to be 16 in the units of U' B' (2^20 is
    // usual; an error of 2^-9 if every B is at its largest) or, where its terms cancel, they have to add up to 1/8
    // (2^-10).  Less is left of tokens far smaller than a later one, or than those before a decay to nothing.  If a
    // token's U' is not finite, zeros of B times it are NaN in all outputs, those before it too.  The zeros of a zero q
    // are right.  (From what is at hand anyway: the outputs as stored for their rows' copies, U' and B' in their first
    // parts.)
    auto apart = [&](const Chunk<DK> &sg, const uint32_t (&uh)[4], float j0, float j1) {
        constexpr uint32_t kAbs = 0x7FFF7FFFu;
        const uint32_t u[4] = {uh[0] & kAbs, uh[1] & kAbs, uh[2] & kAbs, uh[3] & kAbs};
        bool bad = false;
#pragma unroll
        for (int n = 0; n < 2; ++n) {
            const uint4 b = sg.B[8 * n + g][t];
            float terms[4] = {};
            mma_f16(terms, u, b.x & kAbs, b.y & kAbs);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int token = 8 * n + 2 * t + (e & 1);
                const float o = fabsf(lo_bf(mine[token][g + 8 * (e >> 1)])), iq = sg.iq[token];
                bad |= isnan(o) || (iq >= kLeastQ && o < least_for(e < 2 ? j0 : j1) * iq && terms[e] < 0.125f);
            }
        }
        return __any_sync(~0u, bad && live);
    };
    // The tokens of chunk c by the definition, in FP32, for chunks whose tokens are too far apart: a token then
    // depends on those before it alone.  7 us a chunk instead of 1.6, so it is to be rare: by chance one of 10^6 rows that start
    // empty, and chunks of an empty state, or a decay to nothing, where tokens that write nothing come before others.  A lane has 2 NT channels of its rows g and g + 8.
    auto one_by_one = [&](int64_t c) {
        __syncwarp();  // the outputs of the product are stored
        rescale(i0, i1);
        const int h = sm.head, hq = h / (p.Hv / p.Hq);  // (from shared memory: no registers over the loop for this)
        const int64_t first = sm.token + c * kC, end = sm.end < first + kC ? sm.end : first + kC;
#pragma unroll 1
        for (int64_t tok = first; tok < end; ++tok) {
            const uint16_t *kp = p.k + tok * p.ks + (int64_t)hq * DK + 2 * t;
            const uint16_t *qp = p.q + tok * p.qs + (int64_t)hq * DK + 2 * t;
            const bool chan = (p.flags & DEP_DELTA_CHANNEL) != 0;
            const float *gp = p.g + tok * p.gs + (chan ? (int64_t)h * DK + 2 * t : h);
            const float a = chan ? 0.f : decay(*gp);
            float kk = 0.f, qq = 0.f, kq = 0.f, k0 = 0.f, k1 = 0.f, q0 = 0.f, q1 = 0.f;
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                const uint32_t kw = *reinterpret_cast<const uint32_t *>(kp + 8 * n);
                const uint32_t qw = *reinterpret_cast<const uint32_t *>(qp + 8 * n);
                const float ax = chan ? decay(gp[8 * n]) : a, ay = chan ? decay(gp[8 * n + 1]) : a;
                const float kx = lo_bf(kw), ky = hi_bf(kw), qx = lo_bf(qw), qy = hi_bf(qw);
                S[n][0] *= ax, S[n][1] *= ay, S[n][2] *= ax, S[n][3] *= ay;
                kk = fmaf(kx, kx, fmaf(ky, ky, kk));
                qq = fmaf(qx, qx, fmaf(qy, qy, qq));
                kq = fmaf(kx, qx, fmaf(ky, qy, kq));
                k0 = fmaf(S[n][0], kx, fmaf(S[n][1], ky, k0));
                q0 = fmaf(S[n][0], qx, fmaf(S[n][1], qy, q0));
                k1 = fmaf(S[n][2], kx, fmaf(S[n][3], ky, k1));
                q1 = fmaf(S[n][2], qx, fmaf(S[n][3], qy, q1));
            }
#pragma unroll
            for (int d = 1; d < 4; d <<= 1) {
                kk += __shfl_xor_sync(~0u, kk, d);
                qq += __shfl_xor_sync(~0u, qq, d);
                kq += __shfl_xor_sync(~0u, kq, d);
                k0 += __shfl_xor_sync(~0u, k0, d);
                q0 += __shfl_xor_sync(~0u, q0, d);
                k1 += __shfl_xor_sync(~0u, k1, d);
                q1 += __shfl_xor_sync(~0u, q1, d);
            }
            float rq = p.scale, rk = 1.f;
            if (p.flags & DEP_DELTA_L2NORM) {
                rk = 1.0f / sqrtf(kk + 1e-6f);
                rq *= 1.0f / sqrtf(qq + 1e-6f);
            }
            kq *= rk * rq;
            const float beta = p.beta[tok * p.bs + h];
            const uint16_t *vp = p.v + tok * p.vs + (int64_t)h * p.Dv + row0 + g;
            const float u0 = beta * ((live ? lo_bf(vp[0]) : 0.f) - k0 * rk);
            const float u1 = beta * ((live ? lo_bf(vp[8]) : 0.f) - k1 * rk);
            if (live && t == 0) {
                uint16_t *o = p.o + tok * p.os + (int64_t)h * p.Dv + row0 + g;
                o[0] = __bfloat16_as_ushort(__float2bfloat16_rn(fmaf(u0, kq, q0 * rq)));
                o[8] = __bfloat16_as_ushort(__float2bfloat16_rn(fmaf(u1, kq, q1 * rq)));
            }
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                const uint32_t kw = *reinterpret_cast<const uint32_t *>(kp + 8 * n);
                const float kx = lo_bf(kw) * rk, ky = hi_bf(kw) * rk;
                S[n][0] = fmaf(u0, kx, S[n][0]), S[n][1] = fmaf(u0, ky, S[n][1]);
                S[n][2] = fmaf(u1, kx, S[n][2]), S[n][3] = fmaf(u1, ky, S[n][3]);
            }
        }
        start_range();
    };
    if (threadIdx.x == 0) {
        sm.head = h;
        sm.token = t0 + from * kC;
        sm.end = t1;
    }
    griddep_wait();  // the chunks; what came before them is done
    for (int c = 0; c < kStages - 1; ++c) {
        fetch(c, 0, kPieces);
        commit();
    }
    constexpr int kPer = (kPieces + NT / 2 - 1) / (NT / 2);
    for (int64_t c = 0; c < chunks; ++c) {
        asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 2) : "memory");
        __syncthreads();
        const Chunk<DK> &sg = sm.stage[c % kStages];
        *reinterpret_cast<uint4 *>(&mine[lane >> 1][8 * (lane & 1)]) = v;
        v = fetch_v(c + 1);
        __syncwarp();
        float U[2][4] = {};
        {  // U^T = V^T T^T - S^T W^T, the part with V
            uint32_t a[4];
            const uint32_t at = (uint32_t)__cvta_generic_to_shared(
                &mine[(lane >> 4) * 8 + (lane & 7)][8 * (lane >> 3 & 1)]);
            asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                         : "=r"(a[0]), "=r"(a[1]), "=r"(a[2]), "=r"(a[3])
                         : "r"(at)
                         : "memory");
            const uint4 b0 = sg.T01[g][t], b1 = sg.T01[8 + g][t];
            const uint2 c0 = sg.T2[g][t], c1 = sg.T2[8 + g][t];
            mma_bf16(U[0], a, c0.x, c0.y);
            mma_bf16(U[1], a, c1.x, c1.y);
            mma_bf16(U[0], a, b0.z, b0.w);
            mma_bf16(U[1], a, b1.z, b1.w);
            mma_bf16(U[0], a, b0.x, b0.y);
            mma_bf16(U[1], a, b1.x, b1.y);
        }
        float X[2][4] = {}, O[2][4] = {};
#pragma unroll
        for (int ks = 0; ks < NT / 2; ++ks) {
            uint32_t ah[4], al[4];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                f16_split2(S[2 * ks + i][0], S[2 * ks + i][1], ah[2 * i], al[2 * i]);
                f16_split2(S[2 * ks + i][2], S[2 * ks + i][3], ah[2 * i + 1], al[2 * i + 1]);
            }
            float(*const d[4])[4] = {&X[0], &O[0], &X[1], &O[1]};
            const int at = (4 * ks + t) ^ (g & 1) << 2;
            const uint4 b[4] = {sg.w[g][at], sg.qp[g][at], sg.w[8 + g][at], sg.qp[8 + g][at]};
            mma_f16x3(d, ah, al, b);
            // The copies among the products: all at once they hold the warps up for 500 cycles.
            fetch(c + kStages - 1, ks * kPer, kPer);
        }
        commit();
        // U' = U / (k's scale), in parts scaled by row: the left operand of B and of K.R
        uint32_t uh[4], ul[4];
        float j0, j1;
        {
#pragma unroll
            for (int n = 0; n < 2; ++n) {
                const float2 iw = ld2(&sg.iw[8 * n + 2 * t]), ik = ld2(&sg.ik[8 * n + 2 * t]);
                // (the scales' product first: X over S's alone may pass FP32's range)
                U[n][0] = fmaf(X[n][0], i0 * -iw.x, U[n][0]) * ik.x;
                U[n][1] = fmaf(X[n][1], i0 * -iw.y, U[n][1]) * ik.y;
                U[n][2] = fmaf(X[n][2], i1 * -iw.x, U[n][2]) * ik.x;
                U[n][3] = fmaf(X[n][3], i1 * -iw.y, U[n][3]) * ik.y;
            }
            const float top0 = row_max(fmaxf(fmaxf(fabsf(U[0][0]), fabsf(U[0][1])), fmaxf(fabsf(U[1][0]), fabsf(U[1][1]))));
            const float top1 = row_max(fmaxf(fmaxf(fabsf(U[0][2]), fabsf(U[0][3])), fmaxf(fabsf(U[1][2]), fabsf(U[1][3]))));
            const float s0 = scale_for(top0, j0), s1 = scale_for(top1, j1);
#pragma unroll
            for (int n = 0; n < 2; ++n) {
                f16_split2(U[n][0] * s0, U[n][1] * s0, uh[2 * n], ul[2 * n]);
                f16_split2(U[n][2] * s1, U[n][3] * s1, uh[2 * n + 1], ul[2 * n + 1]);
            }
        }
        float Y[2][4] = {};  // U^T B^T
        {
            float(*const d[2])[4] = {&Y[0], &Y[1]};
            const uint4 b[2] = {sg.B[g][t], sg.B[8 + g][t]};
            mma_f16x3(d, uh, ul, b);
        }
        // The update's products, U^T (K.R): kTiles tiles of eight channels at a time, the next ones before the sums of
        // these, and the first before O, which has to wait for Y.
        constexpr int kTiles = 4;
        const int sw = t ^ (g >> 1 & 3);
        float D[2][kTiles][4];
        auto products = [&](int n, float (&d2)[kTiles][4]) {
#pragma unroll
            for (int i = 0; i < kTiles; ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    d2[i][e] = 0.f;
            float(*const d[kTiles])[4] = {&d2[0], &d2[1], &d2[2], &d2[3]};
            const uint4 b[kTiles] = {sg.kr[8 * n + g][sw], sg.kr[8 * n + 8 + g][sw], sg.kr[8 * n + 16 + g][sw],
                                     sg.kr[8 * n + 24 + g][sw]};
            mma_f16x3(d, uh, ul, b);
        };
        products(0, D[0]);
        // O = Q.P S^T + U' B', each with its scales
        const float o0 = i0 * (1.f / kUnO), o1 = i1 * (1.f / kUnO), y0 = j0 * (kUnB / kUnO), y1 = j1 * (kUnB / kUnO);
        const float least0 = least_for(j0), least1 = least_for(j1);
        bool off = false;  // an output that apart() has to look at
#pragma unroll
        for (int n = 0; n < 2; ++n) {
            O[n][0] = fmaf(Y[n][0], y0, O[n][0] * o0);
            O[n][1] = fmaf(Y[n][1], y0, O[n][1] * o0);
            O[n][2] = fmaf(Y[n][2], y1, O[n][2] * o1);
            O[n][3] = fmaf(Y[n][3], y1, O[n][3] * o1);
            off |= !(fabsf(O[n][0]) >= least0) || !(fabsf(O[n][1]) >= least0) || !(fabsf(O[n][2]) >= least1) ||
                   !(fabsf(O[n][3]) >= least1);
        }
        // O^T [rows][tokens] -> [token][rows]: four transposed 8 x 8 blocks, then 32 bytes a token
        uint32_t r[4];
#pragma unroll
        for (int n = 0; n < 2; ++n) {
            const float2 iq = ld2(&sg.iq[8 * n + 2 * t]);
            asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r[2 * n]) : "f"(O[n][1] * iq.y), "f"(O[n][0] * iq.x));
            asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r[2 * n + 1]) : "f"(O[n][3] * iq.y), "f"(O[n][2] * iq.x));
        }
        const uint32_t at = (uint32_t)__cvta_generic_to_shared(
            &mine[(lane >> 4) * 8 + (lane & 7)][8 * (lane >> 3 & 1)]);  // over V
        asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(r[0]),
                     "r"(r[1]), "r"(r[2]), "r"(r[3])
                     : "memory");
        __syncwarp();
        const int64_t tok = (from + c) * kC + (lane >> 1);
        if (live && tok < len)
            *reinterpret_cast<uint4 *>(p.o + (t0 + tok) * p.os + (int64_t)h * p.Dv + row0 + 8 * (lane & 1)) =
                *reinterpret_cast<const uint4 *>(&mine[lane >> 1][8 * (lane & 1)]);
        {  // S <- S diag(P_15) + U^T (K.R)
            if (__any_sync(~0u, (off && live) || j0 > 0x1p60f * i0 || j1 > 0x1p60f * i1)) {
                if (apart(sg, uh, j0, j1)) {
                    one_by_one(c);
                    continue;
                }
                // U beyond what S's scales leave room for: make room
                rescale(j0 > 0x1p60f * i0 ? fmaxf(0x1p60f * i0 / j0, 0x1p-126f) : 1.f,
                        j1 > 0x1p60f * i1 ? fmaxf(0x1p60f * i1 / j1, 0x1p-126f) : 1.f);
            }
            const float f0 = j0 * r0, f1 = j1 * r1;
            float m0 = 0.f, m1 = 0.f;
#pragma unroll
            for (int n = 0; n < NT; n += kTiles) {
                if (n + kTiles < NT)
                    products(n + kTiles, D[(n / kTiles + 1) & 1]);
#pragma unroll
                for (int i = 0; i < kTiles; ++i) {
                    const float2 a = ld2(&sg.last[8 * (n + i) + 2 * t]);
                    float(&s)[4] = S[n + i];
                    const float(&d)[4] = D[(n / kTiles) & 1][i];
                    s[0] = fmaf(d[0], f0, s[0] * a.x);
                    s[1] = fmaf(d[1], f0, s[1] * a.y);
                    s[2] = fmaf(d[2], f1, s[2] * a.x);
                    s[3] = fmaf(d[3], f1, s[3] * a.y);
                    m0 = max3_abs(m0, s[0], s[1]);
                    m1 = max3_abs(m1, s[2], s[3]);
                }
            }
            keep_range(m0, m1);
        }
        __syncwarp();
    }
#pragma unroll
    for (int n = 0; n < NT; ++n)
        if (live) {
            *reinterpret_cast<float2 *>(p.s_out + sbase + (int64_t)(row0 + g) * DK + 8 * n + 2 * t) =
                make_float2(S[n][0] * i0, S[n][1] * i0);
            *reinterpret_cast<float2 *>(p.s_out + sbase + (int64_t)(row0 + g + 8) * DK + 8 * n + 2 * t) =
                make_float2(S[n][2] * i1, S[n][3] * i1);
        }
}

template <int DK, bool CHAN>
cudaError_t chunk_launch(DeltaParams p, int64_t bytes, cudaStream_t s)
{
    static std::atomic<uint64_t> devices[2] = {{0}, {0}};
    cudaError_t e = set_smem_attr(delta_prepare_kernel<DK, CHAN>, devices[0]);
    if (e == cudaSuccess)
        e = set_smem_attr(delta_state_kernel<DK>, devices[1]);
    int dev = 0, sms = 0;
    if (e == cudaSuccess)
        e = cudaGetDevice(&dev);
    if (e == cudaSuccess)
        e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    const int64_t all = p.tokens / kC + p.n_seq,
                  most = std::min<int64_t>(bytes / (p.Hv * (int64_t)sizeof(Chunk<DK>)), INT32_MAX / p.Hv);  // of a launch
    const int64_t states = (int64_t)((p.Dv + kRows - 1) / kRows) * p.Hv * p.n_seq;
    if (states > INT32_MAX)
        return cudaErrorInvalidConfiguration;
    for (p.chunk0 = 0; e == cudaSuccess && p.chunk0 < all; p.chunk0 += p.n_chunks) {
        p.n_chunks = all - p.chunk0 < most ? all - p.chunk0 : most;
        p.flags = p.n_chunks * p.Hv <= 2 * sms ? p.flags | kEarly : p.flags & ~kEarly;
        delta_prepare_kernel<DK, CHAN><<<(unsigned)(p.n_chunks * p.Hv), kPrep, sizeof(PrepShared<DK, CHAN>), s>>>(p);
        e = cudaGetLastError();
        if (e == cudaSuccess) {
            cudaLaunchAttribute attr{};
            attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
            attr.val.programmaticStreamSerializationAllowed = 1;
            cudaLaunchConfig_t cfg{};
            cfg.gridDim = dim3((unsigned)states);
            cfg.blockDim = dim3(32 * kStateWarps);
            cfg.dynamicSmemBytes = sizeof(StateShared<DK>);
            cfg.stream = s;
            cfg.attrs = &attr;
            cfg.numAttrs = 1;
            e = cudaLaunchKernelEx(&cfg, delta_state_kernel<DK>, p);
        }
    }
    return e;
}

// What dep_delta_workspace asks for at most.  A pass over part of the chunks has fewer sequences at work at once:
// 8192 tokens of 96 heads in 4 ragged sequences take 1405 us in one pass (1.4 GB), with 1 GiB 1613, 512 MiB 1729 and
// 256 MiB 1812.
constexpr int64_t kMostWorkspace = 2ll << 30;

// Chunks for sequences of eight tokens and more on average: a chunk costs the same whether it holds one token or
// sixteen, while the recurrent kernel pays by the token.  Measured with 128 channels, 6, 8 and 12 tokens a sequence:
// 64 sequences of 96 heads 343, 421 and 586 us token by token, 349, 352 and 358 by chunks; 4 of them 25, 30, 41 and
// 31, 31, 31; one of 32 heads 7, 8, 11 and 12, 12, 12.
bool in_chunks(int64_t tokens, int64_t n_seq) { return n_seq > 0 && tokens >= 8 * n_seq; }

template <int DK>
cudaError_t delta_launch(const DeltaParams &p, int64_t bytes, cudaStream_t s)
{
    if (in_chunks(p.tokens, p.n_seq) && bytes >= p.Hv * (int64_t)sizeof(Chunk<DK>))
        return p.flags & DEP_DELTA_CHANNEL ? chunk_launch<DK, true>(p, bytes, s) : chunk_launch<DK, false>(p, bytes, s);
    return (int64_t)p.n_seq * p.Hv * p.Dv < 32768 ? recurrent_launch<DK, 2>(p, s) : recurrent_launch<DK, 4>(p, s);
}

dep_status_t delta_entry(const dep_delta_args_t *a, void *stream)
{
    if (!a || a->tokens < 0 || a->n_seq < 0 || a->n_states < 0 || a->Hq < 1 || a->Hv < 1 || a->Hv % a->Hq != 0 ||
        (a->flags & ~(DEP_DELTA_CHANNEL | DEP_DELTA_L2NORM)) != 0 || a->workspace_bytes < 0 ||
        (a->workspace_bytes > 0 && !a->workspace))
        return DEP_ERR_INVALID_ARG;
    if ((a->Dk != 64 && a->Dk != 128) || a->Dv < 16 || a->Dv > 256 || a->Dv % 16 != 0)
        return DEP_ERR_UNSUPPORTED;
    if (a->n_seq == 0)
        return a->tokens == 0 ? DEP_OK : DEP_ERR_INVALID_ARG;
    if (!a->cu_seqlens && a->tokens % a->n_seq != 0)
        return DEP_ERR_INVALID_ARG;
    const bool chan = (a->flags & DEP_DELTA_CHANNEL) != 0;
    if (!a->state_out || (a->tokens > 0 && (!a->q || !a->k || !a->v || !a->g || !a->beta || !a->o)))
        return DEP_ERR_INVALID_ARG;
    if (!a->slots && a->n_states < a->n_seq)
        return DEP_ERR_INVALID_ARG;
    const int64_t T = a->tokens, qk = (int64_t)a->Hq * a->Dk, hv = (int64_t)a->Hv * a->Dv,
                  gc = chan ? (int64_t)a->Hv * a->Dk : a->Hv;
    if (T > 0 && (a->q_stride < qk || a->k_stride < qk || a->v_stride < hv || a->o_stride < hv || a->g_stride < gc ||
                  a->beta_stride < a->Hv))
        return DEP_ERR_INVALID_ARG;
    const int64_t sb = (int64_t)a->Hv * a->Dv * a->Dk * 4;
    const Rows q{a->q, 2 * qk, 2 * a->q_stride, T}, k{a->k, 2 * qk, 2 * a->k_stride, T},
        v{a->v, 2 * hv, 2 * a->v_stride, T}, o{a->o, 2 * hv, 2 * a->o_stride, T},
        g{a->g, 4 * gc, 4 * a->g_stride, T}, b{a->beta, 4 * (int64_t)a->Hv, 4 * a->beta_stride, T},
        si{a->state_in, sb, sb, a->state_in ? a->n_states : 0}, so{a->state_out, sb, sb, a->n_states},
        w{a->workspace, a->workspace_bytes, a->workspace_bytes, 1};
    if (!q.aligned(16) || !k.aligned(16) || !v.aligned(16) || !o.aligned(16) || !g.aligned(chan ? 16 : 4) ||
        !b.aligned(4) || !si.aligned(16) || !so.aligned(16) || !aligned(a->cu_seqlens, 4) || !aligned(a->slots, 4) || !aligned(a->workspace, 16))
        return DEP_ERR_MISALIGNED;
    for (const Rows *in : {&q, &k, &v, &g, &b})
        if (overlap(o, *in) || overlap(so, *in))
            return DEP_ERR_INVALID_ARG;
    if (a->workspace_bytes > 0)
        for (const Rows *t : {&q, &k, &v, &g, &b, &o, &si, &so})
            if (overlap(w, *t))
                return DEP_ERR_INVALID_ARG;
    if (overlap(o, so) || overlap(o, si) || (overlap(so, si) && a->state_in != a->state_out))
        return DEP_ERR_INVALID_ARG;
    DeltaParams p;
    p.q = static_cast<const uint16_t *>(a->q);
    p.k = static_cast<const uint16_t *>(a->k);
    p.v = static_cast<const uint16_t *>(a->v);
    p.g = a->g;
    p.beta = a->beta;
    p.s_in = a->state_in;
    p.s_out = a->state_out;
    p.o = static_cast<uint16_t *>(a->o);
    p.cu = a->cu_seqlens;
    p.slots = a->slots;
    p.qs = a->q_stride;
    p.ks = a->k_stride;
    p.vs = a->v_stride;
    p.gs = a->g_stride;
    p.bs = a->beta_stride;
    p.os = a->o_stride;
    p.tokens = T;
    p.n_states = a->n_states;
    p.n_seq = a->n_seq;
    p.Hq = a->Hq;
    p.Hv = a->Hv;
    p.Dv = a->Dv;
    p.flags = a->flags;
    p.scale = a->scale;
    p.chunks = static_cast<uint8_t *>(a->workspace);
    p.chunk0 = p.n_chunks = 0;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const cudaError_t e = a->Dk == 128 ? delta_launch<128>(p, a->workspace_bytes, s) : delta_launch<64>(p, a->workspace_bytes, s);
    if (e != cudaSuccess) {
        cudaGetLastError();
        return e == cudaErrorInvalidConfiguration ? DEP_ERR_UNSUPPORTED : DEP_ERR_CUDA;
    }
    return DEP_OK;
}

}  // namespace
}  // namespace dep

extern "C" dep_status_t dep_delta_workspace(const dep_delta_args_t *a, int64_t *bytes)
{
    if (!a || !bytes || a->tokens < 0 || a->n_seq < 0 || a->Hv < 1)
        return DEP_ERR_INVALID_ARG;
    *bytes = 0;
    const int64_t chunk = a->Hv * (int64_t)(a->Dk == 128 ? sizeof(dep::Chunk<128>) : sizeof(dep::Chunk<64>));
    if (dep::in_chunks(a->tokens, a->n_seq))
        *bytes = std::max(chunk, std::min((a->tokens / dep::kC + a->n_seq) * chunk, dep::kMostWorkspace));
    return DEP_OK;
}

extern "C" dep_status_t dep_delta_rule(const dep_delta_args_t *args, void *stream)
{
    return dep::delta_entry(args, stream);
}
