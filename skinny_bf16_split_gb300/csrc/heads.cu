// heads.cu -- RMS norm of each head of q and k with the rotary position in the same
// pass, and keys and values appended to a paged cache on the way.
//
//     y = x * rstd * w,  rstd = 1 / sqrt(mean(x^2) + eps)
//     (a, b) <- amplitude * (a cos u - b sin u, b cos u + a sin u),  u = position * freq
//
// A head is held by D / 16 neighbouring lanes, sixteen channels each: eight from the first half of
// the rotated channels and the same eight of the second (or sixteen neighbours), so both partners of
// every pair are in one lane and the rotation needs no exchange; the sum of squares is the only one.
// (Eight channels a lane where D or the rotated part is no multiple of 16.)
//
// Angles.  A frequency becomes a 64-bit fraction of a turn, f / 2 pi modulo 1, once a
// block; times the position modulo 2^64 it is the angle without any reduction, to
// 2^-53 of position * f (what FP64 holds of f / 2 pi) however far the position, and then rounded
// to FP32.  A block works the angles of a few tokens out at once, for all their heads.
//
// Bound: DRAM, each byte read once and written once; close behind it the instructions: of 8 channels
// a lane 110 for eight, of 16 about 120 for sixteen (8192 tokens of 96 and 8 heads of 128 channels 116 us
// with eight, 79 with sixteen).  Many tasks a warp go through shared memory, three in flight and one at
// work without registers for them: 73.3 us, 88 % of the copy rate, the issue slots 69 % busy; where that was measured
// to pay is at heads_launch.  8192 tokens into the cache 17.5 us (nine tasks a warp, one ahead, three rounds of angles and
// a barrier each; 22 % of DRAM, 56 % of the issue slots), one token 2.8 (launch, one load, one store).
#include <cuda_bf16.h>

#include <math.h>

#include <algorithm>
#include <type_traits>

#include "internal.h"
#include "layer.h"
#include "ptx.cuh"

namespace dep {
namespace {

constexpr int kThreads = 256;
constexpr int kBlocks = 3;    // of an SM
constexpr int kMostTokens = 16;
constexpr int kStages = 4;    // tasks of a warp in flight, where it has many
constexpr int kTokens = 4;    // whose angles a block has room for, of the widest heads

struct HeadsParams {
    const uint16_t *q, *k, *v, *qw, *kw;
    const double *freqs;
    const int32_t *positions, *slots;
    uint16_t *q_out, *k_out, *kc, *vc;  // k_out or the caches
    int64_t qs, ks, vs, qos, kos;
    int64_t kps, kss, khs, vps, vss, vhs;
    int64_t tokens, n_pages;
    int32_t Hq, Hk, D, rot, first, page;
    int32_t at_once, tasks;  // tokens at once; groups of heads of a token, a warp each
    float eps, amplitude;
};

__device__ __forceinline__ float lo16(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float hi16(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }
__device__ __forceinline__ uint32_t pack16(float lo, float hi)
{
    const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&v);
}

// Two FP32 operations at once.
struct Two {
    uint64_t v;
    __device__ Two() {}
    __device__ Two(float a, float b) { asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "f"(a), "f"(b)); }
    __device__ void apart(float &a, float &b) const { asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v)); }
};
__device__ __forceinline__ Two mul(Two a, Two b)
{
    Two r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
    return r;
}
__device__ __forceinline__ Two sub(Two a, Two b)
{
    Two r;
    asm("sub.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
    return r;
}
__device__ __forceinline__ Two fma(Two a, Two b, Two c)
{
    Two r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
    return r;
}

// A lane's N channels: N / 2 pairs (a, b), two at once.
template <int N>
struct Pairs {
    Two a[N / 4], b[N / 4];
};

// The same as they are in memory: N bytes at o1 and N at o2.
template <int N>
struct Lane {
    uint32_t w[N / 2];
    using Part = typename std::conditional<N == 16, uint4, uint2>::type;
    // On the way through shared memory: the lanes' first halves, then their second ones.
    static __device__ void fetch(Part *to, const uint16_t *p, int o1, int o2)
    {
        const uint32_t at = smem_u32(to);
        static_assert(N == 16, "copies of 16 bytes");
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(at), "l"(p + o1) : "memory");
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(at + 32 * N), "l"(p + o2) : "memory");
    }
    __device__ void arrive(const Part *from)
    {
        *reinterpret_cast<Part *>(w) = from[0];
        *reinterpret_cast<Part *>(w + N / 4) = from[32];
    }
    __device__ void load(const uint16_t *p, int o1, int o2)
    {
        *reinterpret_cast<Part *>(w) = *reinterpret_cast<const Part *>(p + o1);
        *reinterpret_cast<Part *>(w + N / 4) = *reinterpret_cast<const Part *>(p + o2);
    }
    __device__ void store(uint16_t *p, int o1, int o2) const
    {
        *reinterpret_cast<Part *>(p + o1) = *reinterpret_cast<const Part *>(w);
        *reinterpret_cast<Part *>(p + o2) = *reinterpret_cast<const Part *>(w + N / 4);
    }
    // Pairs of neighbours, or of the first half of the channels and the second.
    template <bool INTERLEAVED>
    __device__ Pairs<N> unpack() const
    {
        Pairs<N> x;
#pragma unroll
        for (int i = 0; i < N / 4; ++i) {
            x.a[i] = INTERLEAVED ? Two(lo16(w[2 * i]), lo16(w[2 * i + 1])) : Two(lo16(w[i]), hi16(w[i]));
            x.b[i] = INTERLEAVED ? Two(hi16(w[2 * i]), hi16(w[2 * i + 1])) : Two(lo16(w[N / 4 + i]), hi16(w[N / 4 + i]));
        }
        return x;
    }
    template <bool INTERLEAVED>
    __device__ void pack(const Pairs<N> &x)
    {
#pragma unroll
        for (int i = 0; i < N / 4; ++i) {
            float a0, a1, b0, b1;
            x.a[i].apart(a0, a1);
            x.b[i].apart(b0, b1);
            w[INTERLEAVED ? 2 * i : i] = INTERLEAVED ? pack16(a0, b0) : pack16(a0, a1);
            w[INTERLEAVED ? 2 * i + 1 : N / 4 + i] = INTERLEAVED ? pack16(a1, b1) : pack16(b0, b1);
        }
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

template <int N, int LPH>
__device__ __forceinline__ float head_squares(const Pairs<N> &x)
{
    Two s(0.0f, 0.0f);
#pragma unroll
    for (int i = 0; i < N / 4; ++i)
        s = fma(x.b[i], x.b[i], fma(x.a[i], x.a[i], s));
    float a, b;
    s.apart(a, b);
    return head_sum<LPH>(a + b);
}

template <int N>
__device__ __forceinline__ void scale(Pairs<N> &x, float f)
{
    const Two f2(f, f);
#pragma unroll
    for (int i = 0; i < N / 4; ++i)
        x.a[i] = mul(x.a[i], f2), x.b[i] = mul(x.b[i], f2);
}

// 1 / rms of a head, applied.  Heads whose squares leave FP32's range (of 2^58 and more, or tiny ones with next to
// no eps) are taken times a power of two.
template <int N, int LPH>
__device__ __forceinline__ void normalise(Pairs<N> &x, float inv_d, float D, float eps)
{
    const float ss = head_squares<N, LPH>(x);
    float rstd = rsqrtf(fmaf(ss, inv_d, eps));
    const bool outside = !(ss < 0x1p120f && fmaf(eps, D, ss) > 0x1p-90f);
    if (__any_sync(~0u, outside)) {
        float top = 0.0f;
#pragma unroll
        for (int i = 0; i < N / 4; ++i) {
            float a, b, c, d;
            x.a[i].apart(a, b);
            x.b[i].apart(c, d);
            top = fmaxf(fmaxf(fmaxf(top, fabsf(a)), fmaxf(fabsf(b), fabsf(c))), fabsf(d));
        }
#pragma unroll
        for (int d = LPH / 2; d; d >>= 1)
            top = fmaxf(top, __shfl_xor_sync(~0u, top, d));
        // 2^-e in two factors that FP32 holds; nothing is rounded on the way up, nor what counts on the way down
        const int e = outside && top > 0.0f && top <= 0x1.fffffep127f ? ilogbf(top) : 0;
        const float f0 = scalbnf(1.0f, -(e / 2)), f1 = scalbnf(1.0f, -(e - e / 2));
        Pairs<N> y = x;
        scale(y, f0);
        scale(y, f1);
        const float sy = head_squares<N, LPH>(y);
        if (e != 0 && sy < 0x1p120f) {  // (a NaN or an infinity stays what it was)
            rstd = rsqrtf(fmaf(sy, inv_d, eps * f0 * f0 * f1 * f1));
            x = y;
        }
    }
    scale(x, rstd);
}

// Block: `at_once` tokens from blockIdx.x * at_once on and every gridDim.x-th such group after them; a warp takes
// 32 / LPH heads of a token at a time, in the order q, k, v.
template <int N, int LPH, bool INTERLEAVED, bool NORM, bool STAGED>
__global__ void __launch_bounds__(kThreads, kBlocks) heads_kernel(const HeadsParams p)
{
    constexpr int HPW = 32 / LPH, W = kThreads / 32;
    // What a lane takes for two pairs at once, lanes side by side: cos, cos, sin, sin of their angles, times the
    // amplitude, for each token; and the weights of q and of k, as a, a, b, b.
    __shared__ float4 turn[2][kTokens * DEP_HEADS_MAX_D / 4];
    __shared__ float4 weights[2][N / 4][LPH];
    using Part = typename Lane<N>::Part;
    __shared__ Part flight[STAGED ? W : 1][kStages][64];  // what each lane has fetched for itself
    __shared__ uint64_t per[DEP_HEADS_MAX_D / 2];  // of a turn a position
    const int tid = threadIdx.x, lane = tid % 32, c = lane % LPH, warp = tid / 32;
    const int keys = p.Hq + p.Hk, heads = keys + (p.vc ? p.Hk : 0), pairs = p.rot / 2, lanes = p.rot / N;
    const bool in = N * c < p.D;
    int o1 = N * c, o2 = N * c + N / 2, pair = -1;
    if (N * c >= p.first && N * c < p.first + p.rot) {
        pair = N / 2 * c - p.first / 2;
        if (!INTERLEAVED)
            o1 = p.first + pair, o2 = o1 + pairs;
    }
    griddep_launch_dependents();
    griddep_wait();  // what comes before may write the inputs, and read or write the outputs
    if (tid < pairs) {
        double t = p.freqs[tid] * 0.15915494309189535;  // 1 / 2 pi
        t -= floor(t);
        per[tid] = __double2ull_rn(t * 18446744073709551616.0);
    }
    if (NORM && tid < 2 * LPH && in) {  // (lane c of the first groups: its own channels)
        const uint16_t *const w = tid < LPH ? p.qw : p.kw;
        Lane<N> own;
#pragma unroll
        for (int i = 0; i < N / 2; ++i)
            own.w[i] = 0x3F803F80u;
        if (w)
            own.load(w, o1, o2);
        const Pairs<N> x = own.template unpack<INTERLEAVED>();
#pragma unroll
        for (int i = 0; i < N / 4; ++i) {
            float4 f;
            x.a[i].apart(f.x, f.y);
            x.b[i].apart(f.z, f.w);
            weights[tid / LPH][i][c] = f;
        }
    }
    const float inv_d = 1.0f / (float)p.D, dim = (float)p.D;

    // This warp's tasks, one after another: token t0 + tok, heads HPW * g on, where t0 is a group's first token.
    const int64_t stride = (int64_t)gridDim.x * p.at_once;
    const int g0 = blockIdx.y * W + warp, step = gridDim.y * W;
    int64_t t0 = (int64_t)blockIdx.x * p.at_once;
    const auto count = [&](int64_t t0) { return (int)min((int64_t)p.at_once, p.tokens - t0); };
    const auto settle = [&](int &tok, int &g, int n) {  // a group past a token's last goes on with the next token
        while (g >= p.tasks && tok < n)
            g -= p.tasks, ++tok;
    };
    const auto source = [&](int64_t t, int h) {
        return h < p.Hq ? p.q + t * p.qs + h * p.D : h < keys ? p.k + t * p.ks + (h - p.Hq) * p.D : p.v + t * p.vs + (h - keys) * p.D;
    };
    int n = count(t0), tok = 0, g = g0, buf = 0;
    settle(tok, g, n);
    // Loads run ahead of the tasks, over the groups' ends: one task in registers, or kStages - 1 of them in shared memory.
    Lane<N> next{};
    const auto load = [&](int64_t t, int g) {
        const int h = HPW * g + lane / LPH;
        if (in && h < heads)
            next.load(source(t, h), o1, o2);
    };
    int64_t f0 = t0;
    int fn = n, ftok = 0, fg = g0, in_stage = 0, out_stage = 0;
    const auto fetch = [&] {
        if constexpr (STAGED) {
            settle(ftok, fg, fn);
            while (ftok >= fn && f0 < p.tokens) {
                f0 += stride;
                fn = f0 < p.tokens ? count(f0) : 0, ftok = 0, fg = g0;
                settle(ftok, fg, fn);
            }
            const int h = HPW * fg + lane / LPH;
            if (f0 < p.tokens && in && h < heads)
                Lane<N>::fetch(&flight[warp][in_stage][lane], source(f0 + ftok, h), o1, o2);
            asm volatile("cp.async.commit_group;" ::: "memory");
            in_stage = in_stage + 1 == kStages ? 0 : in_stage + 1;
            fg += step;
        }
    };
    if constexpr (STAGED) {
#pragma unroll
        for (int i = 0; i + 1 < kStages; ++i)
            fetch();
    } else if (tok < n)
        load(t0 + tok, g);
    __syncthreads();  // the frequencies
    for (; t0 < p.tokens; t0 += stride, buf ^= 1) {
        n = count(t0);
        for (int i = tid; i < n * pairs; i += kThreads) {
            const int j = i / pairs, k = i - j * pairs;
            const uint64_t u = per[k] * (uint64_t)(int64_t)p.positions[t0 + j];
            float s, co;
            sincospif((float)(int32_t)(u >> 32) * 0x1p-31f, &s, &co);
            const int l = k / (N / 2), m = k % (N / 2);
            float *const at = reinterpret_cast<float *>(&turn[buf][j * (pairs / 2) + m / 2 * lanes + l]) + (m & 1);
            at[0] = co * p.amplitude;
            at[2] = s * p.amplitude;
        }
        __syncthreads();  // (the other buffer is read for the tokens before, done where this one's is written again)
        while (tok < n) {
            Lane<N> now = next;
            const int h = HPW * g + lane / LPH, at = tok;
            const bool values = HPW * g >= keys;  // all of the warp's heads
            g += step;
            settle(tok, g, n);
            if constexpr (STAGED) {
                fetch();
                asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 1) : "memory");
                if (in && h < heads)
                    now.arrive(&flight[warp][out_stage][lane]);
                out_stage = out_stage + 1 == kStages ? 0 : out_stage + 1;
            } else if (tok < n)
                load(t0 + tok, g);
            else if (t0 + stride < p.tokens) {  // the first task among the next tokens
                int tok1 = 0, g1 = g0;
                const int n1 = count(t0 + stride);
                settle(tok1, g1, n1);
                if (tok1 < n1)
                    load(t0 + stride + tok1, g1);
            }
            if (!values) {
                Pairs<N> x = now.template unpack<INTERLEAVED>();
                if (NORM) {
                    normalise<N, LPH>(x, inv_d, dim, p.eps);
#pragma unroll
                    for (int i = 0; i < N / 4; ++i) {
                        const float4 f = weights[h >= p.Hq][i][c];
                        x.a[i] = mul(x.a[i], Two(f.x, f.y)), x.b[i] = mul(x.b[i], Two(f.z, f.w));
                    }
                }
                if (pair >= 0)
#pragma unroll
                    for (int i = 0; i < N / 4; ++i) {
                        const float4 f = turn[buf][at * (pairs / 2) + i * lanes + pair / (N / 2)];
                        const Two cos(f.x, f.y), sin(f.z, f.w), a = x.a[i];
                        x.a[i] = sub(mul(a, cos), mul(x.b[i], sin));
                        x.b[i] = fma(x.b[i], cos, mul(a, sin));
                    }
                if (h < keys)
                    now.template pack<INTERLEAVED>(x);
            }
            if (!in || h >= heads)
                continue;
            const int64_t t = t0 + at;
            if (h < p.Hq)
                now.store(p.q_out + t * p.qos + h * p.D, o1, o2);
            else if (!p.kc)
                now.store(p.k_out + t * p.kos + (h - p.Hq) * p.D, o1, o2);
            else {
                const int32_t slot = p.slots[t], pg = slot / p.page, place = slot - pg * p.page;
                if (slot < 0 || pg >= p.n_pages)
                    continue;
                if (h < keys)
                    now.store(p.kc + pg * p.kps + place * p.kss + (h - p.Hq) * p.khs, o1, o2);
                else
                    now.store(p.vc + pg * p.vps + place * p.vss + (h - keys) * p.vhs, o1, o2);
            }
        }
        if (t0 + stride < p.tokens) {
            tok = 0, g = g0;
            settle(tok, g, count(t0 + stride));
        }
    }
}

template <int N, int LPH, bool INTERLEAVED, bool NORM>
cudaError_t heads_launch(HeadsParams p, cudaStream_t s)
{
    int dev = 0, sms = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess)
        e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess)
        return e;
    constexpr int HPW = 32 / LPH, W = kThreads / 32;
    const int heads = p.Hq + p.Hk + (p.vc ? p.Hk : 0);
    p.tasks = (heads + HPW - 1) / HPW;
    // The tokens in rounds of equal size over all blocks; a token's heads are spread over blocks while there are
    // too few tokens (each block works the angles out anew).
    const int64_t most = (int64_t)kBlocks * sms;
    const int64_t room = p.rot ? std::min(kTokens * DEP_HEADS_MAX_D / p.rot, kMostTokens) : kMostTokens,
                  rounds = (p.tokens + most * room - 1) / (most * room);
    p.at_once = (int)((p.tokens + most * rounds - 1) / (most * rounds));
    const int64_t groups = (p.tokens + p.at_once - 1) / p.at_once, x = std::min(groups, most);
    const int y = (int)std::min<int64_t>((p.tasks + W - 1) / W, (most + x - 1) / x);
    cudaLaunchAttribute attr{};  // starts early, and waits inside
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)x, (unsigned)y);
    cfg.blockDim = dim3(kThreads);
    cfg.stream = s;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    // Many tasks for a warp pay for the way through shared memory, where all channels are rotated by halves in all lanes and
    // a token has many heads.  104 heads of 128, by tasks a warp: 6 of them 12.8 us against 12.9 in registers, 13 19.7 against 20.8,
    // 26 34.6 against 37.6, 59 73.3 against 79.3; 72 of 64: 12 22.2 against 21.9, 16 27.0 against 27.7, 40 52.5 against 57.5.
    // With few heads a token, the angles' barriers are what counts: 24 of 64, 40 tasks a warp, 62.4 against 62.7, 16 of 128 into
    // the cache, 54 a warp, 84.7 against 82.6.  By neighbours (40 a warp) it takes 73.6 against 59.3, half of the channels 61.1
    // against 58.8, heads of 256 64.4 against 62.5.
    if constexpr (N == 16 && LPH <= 8 && !INTERLEAVED)
        if (p.rot == N * LPH && p.tasks >= 9 && rounds * p.at_once * p.tasks / ((int64_t)W * y) >= 16)
            return cudaLaunchKernelEx(&cfg, heads_kernel<N, LPH, INTERLEAVED, NORM, true>, p);
    return cudaLaunchKernelEx(&cfg, heads_kernel<N, LPH, INTERLEAVED, NORM, false>, p);
}

template <int N, int LPH>
cudaError_t heads_dispatch(const HeadsParams &p, uint32_t flags, cudaStream_t s)
{
    const bool n = flags & DEP_HEADS_NORM;
    if (flags & DEP_HEADS_INTERLEAVED)
        return n ? heads_launch<N, LPH, true, true>(p, s) : heads_launch<N, LPH, true, false>(p, s);
    return n ? heads_launch<N, LPH, false, true>(p, s) : heads_launch<N, LPH, false, false>(p, s);
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
    const bool wide = a->D % 16 == 0 && a->rot % 16 == 0 && a->first % 16 == 0;  // sixteen channels a lane
    const cudaError_t e = a->D <= 64    ? wide ? heads_dispatch<16, 4>(p, a->flags, s) : heads_dispatch<8, 8>(p, a->flags, s)
                          : a->D <= 128 ? wide ? heads_dispatch<16, 8>(p, a->flags, s) : heads_dispatch<8, 16>(p, a->flags, s)
                          : wide        ? heads_dispatch<16, 16>(p, a->flags, s)
                                        : heads_dispatch<8, 32>(p, a->flags, s);
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
