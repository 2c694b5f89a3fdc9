// attention.cu -- attention of new tokens over a paged cache.
//
// One warp for each token and query head, one position at a time with the running maximum and sum of a
// softmax.
#include <cuda_bf16.h>

#include <math.h>

#include <algorithm>

#include "internal.h"
#include "layer.h"

namespace dep {
namespace {

constexpr int kTreeMost = 64;  // tokens of a sequence that a tree's words name

struct AttnParams {
    const uint16_t *q, *kc, *vc;
    const int32_t *table, *lens, *cu;
    const uint64_t *tree;
    uint16_t *o;
    float *lse;
    int64_t qs, os, kps, kss, khs, vps, vss, vhs, ts;
    int64_t tokens, n_pages;
    int32_t n_seq, Hq, Hk, page, width;
    float scale;
};

__device__ __forceinline__ int64_t seq_start(const AttnParams &p, int s)
{
    if (!p.cu)
        return p.tokens / p.n_seq * s;
    const int64_t t = p.cu[s];
    return t < 0 ? 0 : t > p.tokens ? p.tokens : t;
}

template <int D>
__global__ void __launch_bounds__(128) rows_kernel(const AttnParams p)
{
    constexpr int E = D / 32;
    const int lane = threadIdx.x & 31;
    const int64_t rows = p.tokens * p.Hq;
    for (int64_t r = blockIdx.x * 4ll + threadIdx.x / 32; r < rows; r += gridDim.x * 4ll) {
        const int64_t t = r / p.Hq;
        const int h = (int)(r % p.Hq), kh = h / (p.Hq / p.Hk);
        int lo = 0, hi = p.n_seq;  // the last sequence that starts at or before t
        while (hi - lo > 1) {
            const int mid = (lo + hi) / 2;
            (seq_start(p, mid) <= t ? lo : hi) = mid;
        }
        const int64_t first = seq_start(p, lo), n = seq_start(p, lo + 1) - first, i = t - first;
        if (i < 0 || i >= n)
            continue;
        const int64_t most = (int64_t)p.width * p.page, len = p.lens[lo] < 0 ? 0 : p.lens[lo] < most ? p.lens[lo] : most;
        float q[E], o[E] = {}, m = -INFINITY, l = 0.0f;
        for (int e = 0; e < E; ++e)
            q[e] = __uint_as_float((uint32_t)p.q[t * p.qs + h * D + lane * E + e] << 16);
        for (int64_t j = 0; j < len; ++j) {
            const int64_t own = j - (len - n);
            if (own >= 0 && (p.tree ? own >= kTreeMost || !(p.tree[t] >> own & 1) : own > i))
                continue;
            const int32_t pg = p.table[lo * p.ts + j / p.page];
            if (pg < 0 || pg >= p.n_pages)
                continue;
            const uint16_t *k = p.kc + pg * p.kps + j % p.page * p.kss + kh * p.khs + lane * E;
            const uint16_t *v = p.vc + pg * p.vps + j % p.page * p.vss + kh * p.vhs + lane * E;
            float x = 0.0f;
            for (int e = 0; e < E; ++e)
                x = fmaf(q[e], __uint_as_float((uint32_t)k[e] << 16), x);
            for (int d = 16; d; d >>= 1)
                x += __shfl_xor_sync(~0u, x, d);
            x *= p.scale;
            if (x == -INFINITY)
                continue;
            const float top = fmaxf(m, x), f = m == top ? 1.0f : expf(m - top), e1 = expf(x - top);
            l = fmaf(l, f, e1);
            for (int e = 0; e < E; ++e)
                o[e] = fmaf(o[e], f, e1 * __uint_as_float((uint32_t)v[e] << 16));
            m = top;
        }
        const float inv = l == 0.0f ? 0.0f : 1.0f / l;
        for (int e = 0; e < E; ++e)
            reinterpret_cast<__nv_bfloat16 *>(p.o)[t * p.os + h * D + lane * E + e] = __float2bfloat16_rn(l == 0.0f ? 0.0f : o[e] * inv);
        if (p.lse && lane == 0)
            p.lse[r] = l == 0.0f ? -INFINITY : m + logf(l);
    }
}

template <int D>
cudaError_t attn_launch(const AttnParams &p, cudaStream_t s)
{
    rows_kernel<D><<<(unsigned)std::min<int64_t>((p.tokens * p.Hq + 3) / 4, 1 << 20), 128, 0, s>>>(p);
    return cudaGetLastError();
}

dep_status_t attn_entry(const dep_attention_args_t *a, void *stream)
{
    if (!a || a->tokens < 0 || a->n_seq < 0 || a->Hq < 1 || a->Hk < 1 || a->Hq % a->Hk != 0 || a->page_size < 1 ||
        a->table_width < 0 || a->n_pages < 0 || a->workspace_bytes < 0 || !(a->scale >= 0.0f) || isinf(a->scale))
        return DEP_ERR_INVALID_ARG;
    if (a->D != 64 && a->D != 128)
        return DEP_ERR_UNSUPPORTED;
    if (a->n_seq == 0)
        return a->tokens == 0 ? DEP_OK : DEP_ERR_INVALID_ARG;
    if (!a->cu_seqlens && a->tokens % a->n_seq != 0)
        return DEP_ERR_INVALID_ARG;
    if (a->tokens == 0)
        return DEP_OK;
    int64_t need = 0;
    if (dep_attention_workspace(a, &need) != DEP_OK)
        return DEP_ERR_UNSUPPORTED;
    const bool cache = a->n_pages > 0 && a->table_width > 0;
    if (!a->q || !a->o || !a->kv_lens || (a->table_width > 0 && !a->page_table) ||
        (cache && (!a->k_cache || !a->v_cache)) || a->workspace_bytes < need || (need > 0 && !a->workspace))
        return DEP_ERR_INVALID_ARG;
    const int64_t T = a->tokens, qn = (int64_t)a->Hq * a->D;
    if (a->q_stride < qn || a->o_stride < qn || a->table_stride < a->table_width)
        return DEP_ERR_INVALID_ARG;
    // Lengths and rows of a sequence in 32 bits.
    if ((int64_t)a->table_width * a->page_size > INT32_MAX - 4096 || T * (int64_t)a->Hq > INT32_MAX - 4096 || a->n_pages > INT32_MAX)
        return DEP_ERR_UNSUPPORTED;
    const CacheRows kc{cache ? a->k_cache : nullptr, 2ll * a->D, {{2 * a->k_page_stride, a->n_pages}, {2 * a->k_slot_stride, a->page_size}, {2 * a->k_head_stride, a->Hk}}},
        vc{cache ? a->v_cache : nullptr, 2ll * a->D, {{2 * a->v_page_stride, a->n_pages}, {2 * a->v_slot_stride, a->page_size}, {2 * a->v_head_stride, a->Hk}}};
    if (!kc.sound() || !vc.sound())
        return DEP_ERR_INVALID_ARG;
    const Rows q{a->q, 2 * qn, 2 * a->q_stride, T}, o{a->o, 2 * qn, 2 * a->o_stride, T},
        lse{a->lse, 4 * T * a->Hq, 0, a->lse ? 1 : 0},
        cu{a->cu_seqlens, 4 * ((int64_t)a->n_seq + 1), 0, a->cu_seqlens ? 1 : 0}, kv{a->kv_lens, 4 * (int64_t)a->n_seq, 0, 1},
        table{a->page_table, 4 * (int64_t)a->table_width, 4 * a->table_stride, a->table_width > 0 ? a->n_seq : 0},
        tree{a->tree, 8 * T, 0, a->tree ? 1 : 0}, w{a->workspace, need, 0, need > 0 ? 1 : 0};
    if (!q.aligned(16) || !o.aligned(16) || !kc.aligned(16) || !vc.aligned(16) || !w.aligned(16) || !tree.aligned(8) ||
        !lse.aligned(4) || !cu.aligned(4) || !kv.aligned(4) || !table.aligned(4))
        return DEP_ERR_MISALIGNED;
    const Rows ks = kc.span(), vs = vc.span();
    for (const Rows *in : {&q, &cu, &kv, &table, &tree, &ks, &vs})
        if (overlap(o, *in) || overlap(lse, *in) || overlap(w, *in))
            return DEP_ERR_INVALID_ARG;
    if (overlap(o, lse) || overlap(o, w) || overlap(lse, w))
        return DEP_ERR_INVALID_ARG;
    AttnParams p{};
    p.q = static_cast<const uint16_t *>(a->q), p.kc = static_cast<const uint16_t *>(a->k_cache), p.vc = static_cast<const uint16_t *>(a->v_cache);
    p.table = a->page_table, p.lens = a->kv_lens, p.cu = a->cu_seqlens, p.tree = a->tree;
    p.o = static_cast<uint16_t *>(a->o), p.lse = a->lse;
    p.qs = a->q_stride, p.os = a->o_stride;
    p.kps = a->k_page_stride, p.kss = a->k_slot_stride, p.khs = a->k_head_stride;
    p.vps = a->v_page_stride, p.vss = a->v_slot_stride, p.vhs = a->v_head_stride;
    p.ts = a->table_stride, p.tokens = T, p.n_pages = cache ? a->n_pages : 0;
    p.n_seq = a->n_seq, p.Hq = a->Hq, p.Hk = a->Hk, p.page = a->page_size, p.width = a->table_width;
    p.scale = a->scale;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const cudaError_t e = a->D == 128 ? attn_launch<128>(p, s) : attn_launch<64>(p, s);
    if (e != cudaSuccess) {
        cudaGetLastError();
        return DEP_ERR_CUDA;
    }
    return DEP_OK;
}

}  // namespace
}  // namespace dep

extern "C" {

dep_status_t dep_attention_workspace(const dep_attention_args_t *a, int64_t *bytes)
{
    if (!a || !bytes || a->tokens < 0 || a->n_seq < 0 || a->Hq < 1 || a->Hk < 1)
        return DEP_ERR_INVALID_ARG;
    *bytes = 0;
    return DEP_OK;
}

dep_status_t dep_paged_attention(const dep_attention_args_t *args, void *stream)
{
    return dep::attn_entry(args, stream);
}

}  // extern "C"
