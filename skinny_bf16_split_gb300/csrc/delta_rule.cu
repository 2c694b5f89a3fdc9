// delta_rule.cu -- the gated delta rule of a delta-attention layer.
//
//     S <- S diag(a),  S <- S + beta (v - S k) k^T,  o = scale S q,   a = exp(g)
//
// S [Dv, Dk] in FP32 for each (sequence, value head).  The rows of S (value
// channels) never meet: any set of rows can go to any warp.
//
// Recurrent kernel.  A group of eight lanes holds a row (Dk / 8 channels a lane,
// in chunks of four so that a group reads 128 consecutive bytes); a warp holds
// 4 * SETS rows.  The two dot products S k and S q are taken of the decayed state
// together, so each token costs one reduction: with u = beta (v - S k),
// o = scale (S q + u (k . q)) and S + u k^T.
// Bound: DRAM, the state read and written once (8 Dk Dv bytes a head).
#include <cuda_bf16.h>

#include "internal.h"
#include "layer.h"

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
};

__device__ __forceinline__ float lo_bf(uint32_t v) { return __uint_as_float(v << 16); }
__device__ __forceinline__ float hi_bf(uint32_t v) { return __uint_as_float(v & 0xFFFF0000u); }

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
    const int slices = (p.Dv + kRecWarps * 4 * SETS - 1) / (kRecWarps * 4 * SETS);
    const int slice = blockIdx.x % slices;
    const int64_t sh = blockIdx.x / slices;
    const int h = (int)(sh % p.Hv), s = (int)(sh / p.Hv);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, l8 = lane & 7;
    const int row0 = (slice * kRecWarps + warp) * 4 * SETS;  // the warp's first row
    if (row0 >= p.Dv)
        return;
    int64_t t0, t1;
    seq_range(p, s, t0, t1);
    const int64_t slot = p.slots ? p.slots[s] : s;
    if (slot < 0 || slot >= p.n_states) {  // padding: zeros out, no state
        for (int64_t t = t0; t < t1; ++t)
            for (int r = lane; r < 4 * SETS; r += 32)
                if (row0 + r < p.Dv)
                    p.o[t * p.os + (int64_t)h * p.Dv + row0 + r] = 0;
        return;
    }
    const int64_t sbase = (slot * p.Hv + h) * (int64_t)p.Dv * DK;
    float4 S[SETS][NV];
#pragma unroll
    for (int i = 0; i < SETS; ++i) {
        const int row = row0 + 4 * i + (lane >> 3);
#pragma unroll
        for (int c = 0; c < NV; ++c)
            S[i][c] = p.s_in && row < p.Dv
                          ? *reinterpret_cast<const float4 *>(p.s_in + sbase + (int64_t)row * DK + 32 * c + 4 * l8)
                          : make_float4(0.f, 0.f, 0.f, 0.f);
    }
    const int hq = h / (p.Hv / p.Hq);
    for (int64_t t = t0; t < t1; ++t) {
        float4 k[NV], q[NV], a[NV];
        float kk = 0.f, qq = 0.f, kq = 0.f;
#pragma unroll
        for (int c = 0; c < NV; ++c) {
            const uint2 kb = *reinterpret_cast<const uint2 *>(p.k + t * p.ks + (int64_t)hq * DK + 32 * c + 4 * l8);
            const uint2 qb = *reinterpret_cast<const uint2 *>(p.q + t * p.qs + (int64_t)hq * DK + 32 * c + 4 * l8);
            k[c] = make_float4(lo_bf(kb.x), hi_bf(kb.x), lo_bf(kb.y), hi_bf(kb.y));
            q[c] = make_float4(lo_bf(qb.x), hi_bf(qb.x), lo_bf(qb.y), hi_bf(qb.y));
            if (p.flags & DEP_DELTA_CHANNEL) {
                const float4 g =
                    *reinterpret_cast<const float4 *>(p.g + t * p.gs + (int64_t)h * DK + 32 * c + 4 * l8);
                a[c] = make_float4(expf(g.x), expf(g.y), expf(g.z), expf(g.w));
            }
        }
        if (!(p.flags & DEP_DELTA_CHANNEL)) {
            const float e = expf(p.g[t * p.gs + h]);
#pragma unroll
            for (int c = 0; c < NV; ++c)
                a[c] = make_float4(e, e, e, e);
        }
#pragma unroll
        for (int c = 0; c < NV; ++c) {
            const float *kp = &k[c].x, *qp = &q[c].x;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                kk = fmaf(kp[j], kp[j], kk);
                qq = fmaf(qp[j], qp[j], qq);
                kq = fmaf(kp[j], qp[j], kq);
            }
        }
#pragma unroll
        for (int d = 4; d; d >>= 1) {
            kk += __shfl_xor_sync(~0u, kk, d);
            qq += __shfl_xor_sync(~0u, qq, d);
            kq += __shfl_xor_sync(~0u, kq, d);
        }
        float rq = p.scale, rk = 1.f;
        if (p.flags & DEP_DELTA_L2NORM) {
            rk = 1.0f / sqrtf(kk + 1e-6f);
            rq *= 1.0f / sqrtf(qq + 1e-6f);
        }
        kq *= rk * rq;
        const float beta = p.beta[t * p.bs + h];
#pragma unroll
        for (int i = 0; i < SETS; ++i) {
            const int row = row0 + 4 * i + (lane >> 3);
            float dk = 0.f, dq = 0.f;
#pragma unroll
            for (int c = 0; c < NV; ++c) {
                float *sp = &S[i][c].x;
                const float *ap = &a[c].x, *kp = &k[c].x, *qp = &q[c].x;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    sp[j] *= ap[j];
                    dk = fmaf(sp[j], kp[j], dk);
                    dq = fmaf(sp[j], qp[j], dq);
                }
            }
#pragma unroll
            for (int d = 4; d; d >>= 1) {
                dk += __shfl_xor_sync(~0u, dk, d);
                dq += __shfl_xor_sync(~0u, dq, d);
            }
            const float v =
                row < p.Dv ? __uint_as_float((uint32_t)p.v[t * p.vs + (int64_t)h * p.Dv + row] << 16) : 0.f;
            const float u = beta * (v - dk * rk), uk = u * rk;
#pragma unroll
            for (int c = 0; c < NV; ++c) {
                float *sp = &S[i][c].x;
                const float *kp = &k[c].x;
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    sp[j] = fmaf(uk, kp[j], sp[j]);
            }
            if (l8 == 0 && row < p.Dv)
                p.o[t * p.os + (int64_t)h * p.Dv + row] =
                    __bfloat16_as_ushort(__float2bfloat16_rn(fmaf(u, kq, dq * rq)));
        }
    }
#pragma unroll
    for (int i = 0; i < SETS; ++i) {
        const int row = row0 + 4 * i + (lane >> 3);
#pragma unroll
        for (int c = 0; c < NV; ++c)
            if (row < p.Dv)
                *reinterpret_cast<float4 *>(p.s_out + sbase + (int64_t)row * DK + 32 * c + 4 * l8) = S[i][c];
    }
}

template <int DK>
cudaError_t recurrent_launch(const DeltaParams &p, cudaStream_t s)
{
    constexpr int SETS = 2;  // 32 rows a block
    const int64_t slices = (p.Dv + kRecWarps * 4 * SETS - 1) / (kRecWarps * 4 * SETS);
    const int64_t blocks = slices * p.Hv * p.n_seq;
    if (blocks > INT32_MAX)
        return cudaErrorInvalidConfiguration;
    delta_recurrent_kernel<DK, SETS><<<(unsigned)blocks, kRecWarps * 32, 0, s>>>(p);
    return cudaGetLastError();
}

dep_status_t delta_entry(const dep_delta_args_t *a, void *stream)
{
    if (!a || a->tokens < 0 || a->n_seq < 0 || a->n_states < 0 || a->Hq < 1 || a->Hv < 1 || a->Hv % a->Hq != 0 ||
        (a->flags & ~(DEP_DELTA_CHANNEL | DEP_DELTA_L2NORM)) != 0)
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
        si{a->state_in, sb, sb, a->state_in ? a->n_states : 0}, so{a->state_out, sb, sb, a->n_states};
    if (!q.aligned(16) || !k.aligned(16) || !v.aligned(16) || !o.aligned(16) || !g.aligned(chan ? 16 : 4) ||
        !b.aligned(4) || !si.aligned(16) || !so.aligned(16) || !aligned(a->cu_seqlens, 4) || !aligned(a->slots, 4))
        return DEP_ERR_MISALIGNED;
    for (const Rows *in : {&q, &k, &v, &g, &b})
        if (overlap(o, *in) || overlap(so, *in))
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
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const cudaError_t e = a->Dk == 128 ? recurrent_launch<128>(p, s) : recurrent_launch<64>(p, s);
    if (e != cudaSuccess) {
        cudaGetLastError();
        return e == cudaErrorInvalidConfiguration ? DEP_ERR_UNSUPPORTED : DEP_ERR_CUDA;
    }
    return DEP_OK;
}

}  // namespace
}  // namespace dep

extern "C" dep_status_t dep_delta_rule(const dep_delta_args_t *args, void *stream)
{
    return dep::delta_entry(args, stream);
}
