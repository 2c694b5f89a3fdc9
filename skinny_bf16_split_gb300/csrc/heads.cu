// heads.cu -- RMS norm of each head of q and k with the rotary position in the same
// pass, and keys and values appended to a paged cache on the way.
//
//     y = x * rstd * w,  rstd = 1 / sqrt(mean(x^2) + eps)
//     (a, b) <- amplitude * (a cos u - b sin u, b cos u + a sin u),  u = position * freq
//
// A head is held by D / 8 neighbouring lanes, eight channels each: four from the first
// half of the rotated channels and the same four of the second (or eight neighbours), so
// both partners of every pair are in one lane and the rotation needs no exchange.  The
// eight lanes' (or 16, 32) sum of squares is the only one.
//
// Angles.  A frequency becomes a 64-bit fraction of a turn, f / 2 pi modulo 1, once a
// thread; times the position modulo 2^64 it is the angle without any reduction, to
// 2^-53 of position * f (what FP64 holds of f / 2 pi) however far the position.  A block
// works the rot / 2 angles of its token out once, for all heads.
//
// Bound: DRAM, each byte read once and written once.
#include <cuda_bf16.h>

#include <math.h>

#include <algorithm>

#include "internal.h"
#include "layer.h"

namespace dep {
namespace {

constexpr int kThreads = 256;

struct HeadsParams {
    const uint16_t *q, *k, *v, *qw, *kw;
    const double *freqs;
    const int32_t *positions, *slots;
    uint16_t *q_out, *k_out, *kc, *vc;  // k_out or the caches
    int64_t qs, ks, vs, qos, kos;
    int64_t kps, kss, khs, vps, vss, vhs;
    int64_t tokens, n_pages;
    int32_t Hq, Hk, D, rot, first, page, passes;  // passes: of kThreads / LPH heads, of a block
    float eps, amplitude;
};

__device__ __forceinline__ float lo16(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float hi16(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }
__device__ __forceinline__ uint32_t pack16(float lo, float hi)
{
    const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&v);
}

// A lane's eight channels as they are in memory: 8 bytes at o1 and 8 at o2.
struct Lane {
    uint32_t w[4];
    __device__ void load(const uint16_t *p, int o1, int o2)
    {
        const uint2 a = *reinterpret_cast<const uint2 *>(p + o1), b = *reinterpret_cast<const uint2 *>(p + o2);
        w[0] = a.x, w[1] = a.y, w[2] = b.x, w[3] = b.y;
    }
    __device__ void store(uint16_t *p, int o1, int o2) const
    {
        *reinterpret_cast<uint2 *>(p + o1) = make_uint2(w[0], w[1]);
        *reinterpret_cast<uint2 *>(p + o2) = make_uint2(w[2], w[3]);
    }
    __device__ void unpack(float (&f)[8]) const
    {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            f[2 * i] = lo16(w[i]), f[2 * i + 1] = hi16(w[i]);
    }
};

template <int LPH>
__device__ __forceinline__ float head_sum(float v)
{
#pragma unroll
    for (int d = LPH / 2; d; d >>= 1)
        v += __shfl_xor_sync(~0u, v, d);
    return v;
}

// 1 / rms of a head, and its channels times what goes with it.  Squares that leave FP32's range
// (heads of 2^58 and more, or tiny ones with next to no eps) are taken of the head times a power of two.
template <int LPH>
__device__ __forceinline__ float head_rstd(float (&x)[8], int D, float eps)
{
    float ss = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i)
        ss = fmaf(x[i], x[i], ss);
    ss = head_sum<LPH>(ss);
    float rstd = rsqrtf(ss / (float)D + eps);
    const bool outside = !(ss < 0x1p120f && fmaf(eps, (float)D, ss) > 0x1p-90f);
    if (__any_sync(~0u, outside)) {
        float top = 0.0f;
#pragma unroll
        for (int i = 0; i < 8; ++i)
            top = fmaxf(top, fabsf(x[i]));
#pragma unroll
        for (int d = LPH / 2; d; d >>= 1)
            top = fmaxf(top, __shfl_xor_sync(~0u, top, d));
        const int e = top > 0.0f && top <= 0x1.fffffep127f ? ilogbf(top) : 0;
        float y[8], sy = 0.0f;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            y[i] = scalbnf(x[i], -e);
            sy = fmaf(y[i], y[i], sy);
        }
        sy = head_sum<LPH>(sy);
        const float ey = scalbnf(scalbnf(eps, -e), -e);  // (2^-2e by steps that FP32 holds)
        if (outside && e != 0 && sy < 0x1p120f) {  // (a NaN or an infinity stays what it was)
            rstd = rsqrtf(sy / (float)D + ey);
#pragma unroll
            for (int i = 0; i < 8; ++i)
                x[i] = y[i];
        }
    }
    return rstd;
}

// Block: token blockIdx.x and every gridDim.x-th after it, `passes` times kThreads / LPH heads from
// blockIdx.y's on, in the order q, k, v.
template <int LPH, bool INTERLEAVED, bool NORM>
__global__ void __launch_bounds__(kThreads) heads_kernel(const HeadsParams p)
{
    constexpr int HPP = kThreads / LPH;
    __shared__ float2 turn[2][DEP_HEADS_MAX_D / 2];  // cos, sin of a token's angles, times the amplitude
    const int tid = threadIdx.x, c = tid % LPH, heads = p.Hq + p.Hk + (p.vc ? p.Hk : 0);
    const int h0 = blockIdx.y * p.passes * HPP + tid / LPH;
    const bool lane = 8 * c < p.D;
    int o1 = 8 * c, o2 = 8 * c + 4, pair = -1;
    if (8 * c >= p.first && 8 * c < p.first + p.rot) {
        pair = 4 * c - p.first / 2;
        if (!INTERLEAVED)
            o1 = p.first + pair, o2 = o1 + p.rot / 2;
    }
    uint64_t per = 0;  // of a turn a position
    if (tid < p.rot / 2) {
        double t = p.freqs[tid] * 0.15915494309189535;  // 1 / 2 pi
        t -= floor(t);
        per = __double2ull_rn(t * 18446744073709551616.0);
    }
    Lane wq{{0x3F803F80u, 0x3F803F80u, 0x3F803F80u, 0x3F803F80u}}, wk = wq;
    if (NORM && lane && p.qw)
        wq.load(p.qw, o1, o2);
    if (NORM && lane && p.kw)
        wk.load(p.kw, o1, o2);

    int buf = 0;
    for (int64_t t = blockIdx.x; t < p.tokens; t += gridDim.x, buf ^= 1) {
        const uint16_t *q = p.q + t * p.qs, *k = p.k + t * p.ks, *v = p.v + t * p.vs;
        const auto source = [&](int h) {
            return h < p.Hq ? q + h * p.D : h < p.Hq + p.Hk ? k + (h - p.Hq) * p.D : v + (h - p.Hq - p.Hk) * p.D;
        };
        Lane next{};
        if (lane && h0 < heads)
            next.load(source(h0), o1, o2);
        int64_t ko = 0, vo = 0;
        bool keep = true;
        if (p.kc) {
            const int32_t slot = p.slots[t];
            const int32_t pg = slot / p.page, at = slot - pg * p.page;
            keep = slot >= 0 && pg < p.n_pages;
            ko = pg * p.kps + at * p.kss;
            vo = pg * p.vps + at * p.vss;
        }
        if (tid < p.rot / 2) {
            const uint64_t u = per * (uint64_t)(int64_t)p.positions[t];
            float s, co;
            sincospif((float)(int32_t)(u >> 32) * 0x1p-31f, &s, &co);
            turn[buf][tid] = make_float2(co * p.amplitude, s * p.amplitude);
        }
        __syncthreads();  // (the other buffer is read by the token before, done where this one's is written again)
        float2 cs[4] = {{1, 0}, {1, 0}, {1, 0}, {1, 0}};
        if (pair >= 0)
#pragma unroll
            for (int i = 0; i < 4; ++i)
                cs[i] = turn[buf][pair + i];
        for (int i = 0, h = h0; i < p.passes; ++i, h += HPP) {
            Lane now = next;
            if (i + 1 < p.passes && lane && h + HPP < heads)
                next.load(source(h + HPP), o1, o2);
            if (h < p.Hq + p.Hk || NORM) {  // (all lanes of a warp take part in a sum)
                float x[8], w[8];
                now.unpack(x);
                if (NORM) {
                    const float rstd = head_rstd<LPH>(x, p.D, p.eps);
                    (h < p.Hq ? wq : wk).unpack(w);
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        x[j] = x[j] * rstd * w[j];
                }
                if (h < p.Hq + p.Hk) {
                    if (pair >= 0)
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            float &a = x[INTERLEAVED ? 2 * j : j], &b = x[INTERLEAVED ? 2 * j + 1 : j + 4];
                            const float a0 = a;
                            a = fmaf(a0, cs[j].x, -(b * cs[j].y));
                            b = fmaf(b, cs[j].x, a0 * cs[j].y);
                        }
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        now.w[j] = pack16(x[2 * j], x[2 * j + 1]);
                }
            }
            if (!lane || h >= heads)
                continue;
            if (h < p.Hq)
                now.store(p.q_out + t * p.qos + h * p.D, o1, o2);
            else if (!p.kc)
                now.store(p.k_out + t * p.kos + (h - p.Hq) * p.D, o1, o2);
            else if (keep) {
                const int hk = h - p.Hq;
                if (hk < p.Hk)
                    now.store(p.kc + ko + hk * p.khs, o1, o2);
                else
                    now.store(p.vc + vo + (hk - p.Hk) * p.vhs, o1, o2);
            }
        }
    }
}

template <int LPH, bool INTERLEAVED, bool NORM>
cudaError_t heads_launch(HeadsParams p, cudaStream_t s)
{
    int dev = 0, sms = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess)
        e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess)
        return e;
    constexpr int HPP = kThreads / LPH;
    const int heads = p.Hq + p.Hk + (p.vc ? p.Hk : 0), all = (heads + HPP - 1) / HPP;
    // A token's heads are spread over blocks only while there are too few tokens to fill the GPU: each
    // block works the angles out anew.
    const int64_t x = std::min<int64_t>(p.tokens, 24ll * sms);
    const int y = (int)std::min<int64_t>(all, (8ll * sms + x - 1) / x);
    p.passes = (all + y - 1) / y;
    heads_kernel<LPH, INTERLEAVED, NORM><<<dim3((unsigned)x, (unsigned)((all + p.passes - 1) / p.passes)), kThreads, 0, s>>>(p);
    return cudaGetLastError();
}

template <int LPH>
cudaError_t heads_dispatch(const HeadsParams &p, uint32_t flags, cudaStream_t s)
{
    const bool n = flags & DEP_HEADS_NORM;
    if (flags & DEP_HEADS_INTERLEAVED)
        return n ? heads_launch<LPH, true, true>(p, s) : heads_launch<LPH, true, false>(p, s);
    return n ? heads_launch<LPH, false, true>(p, s) : heads_launch<LPH, false, false>(p, s);
}

dep_status_t heads_entry(const dep_heads_args_t *a, bool append, void *stream)
{
    if (!a || a->tokens < 0 || a->Hq < 0 || a->Hk < 0 || a->D < 1 || a->rot < 0 || a->first < 0 ||
        a->first > a->D - a->rot || (a->flags & ~(DEP_HEADS_INTERLEAVED | DEP_HEADS_NORM)) != 0 ||
        !isfinite(a->amplitude))
        return DEP_ERR_INVALID_ARG;
    const bool norm = (a->flags & DEP_HEADS_NORM) != 0;
    if (norm ? !(a->eps >= 0.0f) || isinf(a->eps) : a->q_weight || a->k_weight)
        return DEP_ERR_INVALID_ARG;
    if (append ? a->Hk < 1 || a->n_pages < 0 || a->page_size < 1 || a->k_out
               : a->Hq < 1 || a->v || a->slots || a->k_cache || a->v_cache)
        return DEP_ERR_INVALID_ARG;
    if ((a->q != nullptr) != (a->Hq > 0 && a->tokens > 0) && a->tokens > 0)
        return DEP_ERR_INVALID_ARG;
    if (a->D % 8 != 0 || a->rot % 8 != 0 || a->first % 8 != 0 || a->D > DEP_HEADS_MAX_D)
        return DEP_ERR_UNSUPPORTED;
    // A head's offset, and a cache's last slot, in 32 bits.
    if (((int64_t)a->Hq + 2 * (int64_t)a->Hk) * a->D > INT32_MAX || (append && a->n_pages > INT32_MAX))
        return DEP_ERR_UNSUPPORTED;
    if (a->tokens == 0)
        return DEP_OK;
    if ((a->Hq > 0) != (a->q_out != nullptr) || (a->rot > 0 && (!a->freqs || !a->positions)) ||
        (append ? !a->k || !a->v || !a->slots || (a->n_pages > 0 && (!a->k_cache || !a->v_cache))
                : (a->Hk > 0) != (a->k != nullptr) || (a->Hk > 0) != (a->k_out != nullptr)))
        return DEP_ERR_INVALID_ARG;
    const int64_t T = a->tokens, qn = (int64_t)a->Hq * a->D, kn = (int64_t)a->Hk * a->D;
    if ((qn && (a->q_stride < qn || a->q_out_stride < qn)) || (kn && a->k_stride < kn) ||
        (append ? a->v_stride < kn : kn && a->k_out_stride < kn))
        return DEP_ERR_INVALID_ARG;
    const Rows q{a->q, 2 * qn, 2 * a->q_stride, qn ? T : 0}, k{a->k, 2 * kn, 2 * a->k_stride, kn ? T : 0},
        v{a->v, 2 * kn, 2 * a->v_stride, append ? T : 0}, qo{a->q_out, 2 * qn, 2 * a->q_out_stride, qn ? T : 0},
        ko{a->k_out, 2 * kn, 2 * a->k_out_stride, append || !kn ? 0 : T},
        qw{a->q_weight, 2 * (int64_t)a->D, 0, a->q_weight ? 1 : 0},
        kw{a->k_weight, 2 * (int64_t)a->D, 0, a->k_weight ? 1 : 0}, f{a->freqs, 4 * (int64_t)a->rot, 0, a->rot ? 1 : 0},
        ps{a->positions, 4 * T, 0, a->rot ? 1 : 0}, sl{a->slots, 4 * T, 0, append ? 1 : 0};
    CacheRows kc{}, vc{};
    if (append && a->n_pages > 0) {
        kc = CacheRows{a->k_cache, 2ll * a->D, {{2 * a->k_page_stride, a->n_pages}, {2 * a->k_slot_stride, a->page_size}, {2 * a->k_head_stride, a->Hk}}};
        vc = CacheRows{a->v_cache, 2ll * a->D, {{2 * a->v_page_stride, a->n_pages}, {2 * a->v_slot_stride, a->page_size}, {2 * a->v_head_stride, a->Hk}}};
        if (!kc.sound() || !vc.sound())
            return DEP_ERR_INVALID_ARG;
    }
    for (const Rows *r : {&q, &k, &v, &qo, &ko, &qw, &kw})
        if (!r->aligned(16))
            return DEP_ERR_MISALIGNED;
    if (!f.aligned(8) || !ps.aligned(4) || !sl.aligned(4) || !kc.aligned(16) || !vc.aligned(16))
        return DEP_ERR_MISALIGNED;
    if (!kc.distinct() || !vc.distinct() || overlap(kc, vc))
        return DEP_ERR_INVALID_ARG;
    // A head is read whole before it is written, so q_out may be q and k_out k; nothing else may meet.
    for (const Rows *in : {&q, &k, &v, &qw, &kw, &f, &ps, &sl}) {
        if (overlap(qo, *in) && !(in == &q && a->q_out == a->q && a->q_out_stride == a->q_stride))
            return DEP_ERR_INVALID_ARG;
        if (overlap(ko, *in) && !(in == &k && a->k_out == a->k && a->k_out_stride == a->k_stride))
            return DEP_ERR_INVALID_ARG;
        if (overlap(kc.span(), *in) || overlap(vc.span(), *in))
            return DEP_ERR_INVALID_ARG;
    }
    if (overlap(qo, ko) || overlap(kc.span(), qo) || overlap(vc.span(), qo))
        return DEP_ERR_INVALID_ARG;
    HeadsParams p{};
    p.q = static_cast<const uint16_t *>(a->q), p.k = static_cast<const uint16_t *>(a->k), p.v = static_cast<const uint16_t *>(a->v);
    p.qw = static_cast<const uint16_t *>(a->q_weight), p.kw = static_cast<const uint16_t *>(a->k_weight);
    p.freqs = a->freqs, p.positions = a->positions, p.slots = a->slots;
    p.q_out = static_cast<uint16_t *>(a->q_out), p.k_out = static_cast<uint16_t *>(a->k_out);
    p.kc = append ? static_cast<uint16_t *>(a->k_cache) : nullptr, p.vc = append ? static_cast<uint16_t *>(a->v_cache) : nullptr;
    p.qs = a->q_stride, p.ks = a->k_stride, p.vs = a->v_stride, p.qos = a->q_out_stride, p.kos = a->k_out_stride;
    p.kps = a->k_page_stride, p.kss = a->k_slot_stride, p.khs = a->k_head_stride;
    p.vps = a->v_page_stride, p.vss = a->v_slot_stride, p.vhs = a->v_head_stride;
    p.tokens = T, p.n_pages = a->n_pages;
    p.Hq = a->Hq, p.Hk = a->Hk, p.D = a->D, p.rot = a->rot, p.first = a->first, p.page = append ? a->page_size : 1;
    p.eps = a->eps, p.amplitude = a->amplitude;
    if (append && a->n_pages == 0) {  // all tokens are padding: q alone is left to do
        if (!a->Hq)
            return DEP_OK;
        p.Hk = 0;
    }
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const cudaError_t e = a->D <= 64    ? heads_dispatch<8>(p, a->flags, s)
                          : a->D <= 128 ? heads_dispatch<16>(p, a->flags, s)
                                        : heads_dispatch<32>(p, a->flags, s);
    if (e != cudaSuccess) {
        cudaGetLastError();
        return DEP_ERR_CUDA;
    }
    return DEP_OK;
}

}  // namespace
}  // namespace dep

extern "C" {

dep_status_t dep_norm_rotate(const dep_heads_args_t *args, void *stream)
{
    return dep::heads_entry(args, false, stream);
}

dep_status_t dep_append_kv(const dep_heads_args_t *args, void *stream)
{
    return dep::heads_entry(args, true, stream);
}

}  // extern "C"
