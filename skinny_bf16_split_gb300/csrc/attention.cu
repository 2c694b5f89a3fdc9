// attention.cu -- attention of new tokens over a paged cache, on tcgen05.
//
//     o = sum_j p_j v_j / sum_j p_j,  p_j = exp2(c (q . k_j) - m),  c = scale log2(e)
//
// in one pass over the keys and values with the running maximum m and sum of a softmax.
//
// Rows.  The n tokens of a sequence and the Hq / Hk query heads that share a key and value head are
// the rows of one product: row r is token r / G, head r % G of the G.  A block takes up to 256 of them
// (two tiles of 128, the MMA's M) against tiles of 128 positions: S = Q K^T into tensor memory, a warp
// group for each tile of rows turns its S into P (BF16, in S's own columns, the MMA's A operand from
// tensor memory) and the MMA adds P V to O, which stays in tensor memory.  With 128 rows or fewer the two groups take
// every other tile of positions and their sums are joined at the end, so that both are at work
// whatever the number of rows.
//
// Work.  Every sequence, key and value head and block of rows is an item of ceil(positions seen / 128)
// tiles; the items' tiles, laid end to end, are cut into equal ranges for the blocks, so contexts
// of any lengths fill the GPU evenly.  A block works its range out from the lengths on the device.  An item that is
// cut leaves FP32 parts with their m and sum in the workspace; a second kernel joins them in order.
//
// Keys and values are gathered by cp.async, 16 bytes a lane, row by row from their pages into the
// 128-byte-swizzled layout that the MMA reads (values as an operand whose N runs along memory), so pages may have any
// size and strides.
#include <cuda_bf16.h>

#include <math.h>

#include <algorithm>

#include "internal.h"
#include "layer.h"
#include "ptx.cuh"

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
    int *status;
    int32_t part_rows;
    struct Cut *cuts;  // of every block
    float2 *part_ml;   // m and sum of a part's rows: [block][2][part_rows]
    float *parts;      // their channels
};

__device__ __forceinline__ int64_t seq_start(const AttnParams &p, int s)
{
    if (!p.cu)
        return p.tokens / p.n_seq * s;
    const int64_t t = p.cu[s];
    return t < 0 ? 0 : t > p.tokens ? p.tokens : t;
}

constexpr int kLeast = 4;        // tiles of a block at least
constexpr int kTile = 128;       // positions of a tile; rows of an MMA
constexpr int kProducers = 128;  // threads that gather
constexpr int kWarps = 13;       // 4 + 4 softmax, 4 producing, 1 issuing MMAs
constexpr int kThreads = 32 * kWarps;
constexpr int kSlotRing = 5 * 32768;  // bytes of keys and values in flight
constexpr int kLag = 2;               // copies in flight behind the one being issued, of each producing thread
constexpr int kMasks = 8;             // tiles whose masks are held
constexpr int kBlockRows = 2 * kTile; // rows of an item
constexpr uint64_t kWaitNs = 1000000000ull;

// What a block leaves for the joining kernel where one of its items goes on in other blocks.
struct Cut {
    int32_t parts;  // of the item; 0: none begins here and goes on
    int32_t seq, kv_head, row0, rows;
    int32_t pad[3];
};

template <int D>
struct Smem {
    static constexpr int kTileBytes = kTile * D * 2;
    static constexpr int kSlots = kSlotRing / kTileBytes;
    uint8_t q[2][kTileBytes];          // rows' tiles; the second also joins the groups' sums
    uint8_t ring[kSlots][kTileBytes];  // keys and values
    uint64_t full[kSlots], empty[kSlots];
    uint64_t q_full, q_empty, joined[2], x_full, x_free, drained;
    uint64_t s_full[2], p_full[2], o_full[2];
    uint32_t masks[kMasks][4];  // positions of a tile that are in the cache
    float ml[2][kTile];         // the second group's m and sum
    int64_t scan[kWarps];
    int64_t begin, left, unit0;  // this block's range, and the units before its first sequence
    int32_t seq, blocks;
    uint32_t tmem;
    int32_t odd[2];  // 1 + the last (even, odd) item with values of new tokens that are not finite
    int32_t dead;    // a wait gave up
};

// ---- a sequence, and the items of a range -----------------------------------------------------

struct Seq {
    int64_t first;  // token
    int32_t n, len, blocks, G;
    __device__ void load(const AttnParams &p, int s)
    {
        first = seq_start(p, s);
        const int64_t m = seq_start(p, s + 1) - first, most = (int64_t)p.width * p.page;
        n = m > 0 ? (int32_t)m : 0;
        const int64_t l = p.lens[s];
        len = (int32_t)(l < 0 ? 0 : l < most ? l : most);
        G = p.Hq / p.Hk;
        blocks = (rows() + kBlockRows - 1) / kBlockRows;
    }
    __device__ int rows() const { return n * G; }
    __device__ int own() const { return len - n; }  // position of the first new token
    // Tiles of block rb of rows: up to the last position that one of them may see, at least one.
    __device__ int tiles(const AttnParams &p, int rb) const
    {
        int end;
        if (p.tree)
            end = len - max(0, n - kTreeMost);
        else
            end = own() + (min(rows(), (rb + 1) * kBlockRows) - 1) / G + 1;
        return max(1, (end + kTile - 1) / kTile);
    }
    __device__ int64_t units(const AttnParams &p) const
    {
        if (n == 0)
            return 0;
        int64_t u = 0;
        if (p.tree)
            u = (int64_t)blocks * tiles(p, 0);
        else
            for (int rb = 0; rb < blocks; ++rb)
                u += tiles(p, rb);
        return u * p.Hk;
    }
};

// The items of a block's range, one after another; every role goes through them by itself.
struct Items {
    Seq q;
    int s, kv_head, rb, t0, t1, T;
    int64_t left, unit;  // of the range; of the item's first tile
    __device__ void tiles(const AttnParams &p)
    {
        T = q.tiles(p, rb);
        t1 = (int)min((int64_t)T, t0 + left);
        left -= t1 - t0;
    }
    // Go to unit `begin` of the units from sequence `seq` on, which starts at unit0.
    __device__ void start(const AttnParams &p, int seq, int64_t unit0, int64_t begin, int64_t count)
    {
        s = seq, left = count, unit = unit0;
        q.load(p, s);
        const int64_t head = q.units(p) / p.Hk, skip = (begin - unit0) / head;
        kv_head = (int)skip;
        unit += skip * head;
        for (rb = 0;; ++rb) {
            T = q.tiles(p, rb);
            if (unit + T > begin)
                break;
            unit += T;
        }
        t0 = (int)(begin - unit);
        tiles(p);
    }
    __device__ bool next(const AttnParams &p)
    {
        if (left <= 0)
            return false;
        unit += T;
        t0 = 0;
        if (++rb == q.blocks) {
            rb = 0;
            if (++kv_head == p.Hk) {
                kv_head = 0;
                do {
                    if (++s >= p.n_seq)
                        return false;
                    q.load(p, s);
                } while (q.n == 0);
            }
        }
        tiles(p);
        return true;
    }
    __device__ int row0() const { return rb * kBlockRows; }
    __device__ int rows() const { return min(kBlockRows, q.rows() - row0()); }
    __device__ bool two() const { return rows() > kTile; }  // both groups on the same tiles of positions
    __device__ int count(int g) const { return two() ? t1 - t0 : (t1 - t0 + 1 - g) / 2; }  // tiles of a group
    __device__ int tile(int g, int i) const { return two() ? t0 + i : t0 + 2 * i + g; }
};

__device__ __forceinline__ int64_t range_begin(int64_t units, int block, int blocks) { return units * block / blocks; }

// The page of position pos and its slot; page -1: not in the cache.
__device__ __forceinline__ int32_t page_of(const AttnParams &p, int s, int pos, int end)
{
    const int32_t pg = pos >= 0 && pos < end ? p.table[s * p.ts + pos / p.page] : -1;
    return pg >= 0 && pg < p.n_pages ? pg : -1;
}

// Bits of the 32 positions from `pos` on that token i of the sequence sees (word: its tree, or null).
__device__ __forceinline__ uint32_t seen32(const AttnParams &p, int own, int i, uint64_t word, int pos)
{
    const int at = pos - own;  // of the first position among the new tokens
    if (at <= -32)
        return ~0u;
    if (!p.tree) {
        const int c = i + 1 - at;
        return c >= 32 ? ~0u : c <= 0 ? 0u : (1u << c) - 1;
    }
    if (at >= 0)
        return at < kTreeMost ? (uint32_t)(word >> at) : 0u;
    return ((1u << -at) - 1) | (uint32_t)(word << -at);
}

// ---- tensor memory ----------------------------------------------------------------------------

__device__ __forceinline__ void tmem_ld32(uint32_t taddr, uint32_t (&v)[32])
{
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
        : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]), "=r"(v[8]),
          "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15]), "=r"(v[16]),
          "=r"(v[17]), "=r"(v[18]), "=r"(v[19]), "=r"(v[20]), "=r"(v[21]), "=r"(v[22]), "=r"(v[23]), "=r"(v[24]),
          "=r"(v[25]), "=r"(v[26]), "=r"(v[27]), "=r"(v[28]), "=r"(v[29]), "=r"(v[30]), "=r"(v[31])
        : "r"(taddr));
}
__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t (&v)[32])
{
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
        "%15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};" ::"r"(taddr),
        "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]),
        "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15]), "r"(v[16]), "r"(v[17]), "r"(v[18]),
        "r"(v[19]), "r"(v[20]), "r"(v[21]), "r"(v[22]), "r"(v[23]), "r"(v[24]), "r"(v[25]), "r"(v[26]), "r"(v[27]),
        "r"(v[28]), "r"(v[29]), "r"(v[30]), "r"(v[31])
        : "memory");
}
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&v)[16])
{
    asm volatile("tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, "
                 "%14, %15, %16};" ::"r"(taddr),
                 "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]),
                 "r"(v[9]), "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
                 : "memory");
}
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// D[tmem] (+)= A[tmem] * B[smem desc], BF16 inputs, FP32 accumulation.
__device__ __forceinline__ void mma_bf16_ta(uint32_t d, uint32_t a, uint64_t bdesc, uint32_t idesc, uint32_t accumulate)
{
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
        "r"(a), "l"(bdesc), "r"(idesc), "r"(accumulate)
        : "memory");
}

// Values as B: N (channels) runs along memory, 64 of them in the 128 bytes of a row; the next 64 are
// kTile rows of 128 bytes further (leading offset), the next eight positions 1024 bytes (stride).
__device__ __forceinline__ uint64_t desc_values(uint32_t saddr)
{
    return (uint64_t)((saddr & 0x3FFFFu) >> 4) | ((uint64_t)(kTile * 128 >> 4) << 16) | ((uint64_t)(1024 >> 4) << 32) |
           ((uint64_t)1 << 46) | ((uint64_t)2 << 61);
}

__device__ __forceinline__ float ex2(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ uint32_t pack16(float lo, float hi)
{
    const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&v);
}
__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src, bool in)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(in ? 16 : 0) : "memory");
}

// Wait for a phase; false if this wait or another one of the block gave up.
template <int D>
__device__ __forceinline__ bool wait(Smem<D> &sm, uint64_t &bar, uint32_t parity, const AttnParams &p, int code)
{
    const uint32_t at = smem_u32(&bar);
    if (mbar_try_wait(at, parity))
        return true;
    const uint64_t t0 = globaltimer_ns();
    for (;;) {
        if (mbar_try_wait(at, parity))
            return true;
        if (*reinterpret_cast<volatile int32_t *>(&sm.dead))
            return false;
        if (globaltimer_ns() - t0 > kWaitNs) {
            record_status(p.status, code);
            *reinterpret_cast<volatile int32_t *>(&sm.dead) = 1;
            return false;
        }
    }
}

// The same for a warp that waits together, and stays together.
template <int D>
__device__ __forceinline__ bool wait_warp(Smem<D> &sm, uint64_t &bar, uint32_t parity, const AttnParams &p, int code)
{
    return __all_sync(~0u, wait(sm, bar, parity, p, code));
}

// ---- producing --------------------------------------------------------------------------------

// Rows of 2 D bytes into a swizzled tile of kTile rows; a warp takes 32 of them, lane l knows row l's
// source (null: zeros).
template <int D>
__device__ __forceinline__ void gather(uint32_t tile, const uint16_t *row, const void *any)
{
    constexpr int CH = D / 8, RPI = 32 / CH;  // chunks of a row; rows an instruction
    const int lane = threadIdx.x & 31, warp = threadIdx.x / 32 & 3, c = lane % CH;
    const uint64_t mine = reinterpret_cast<uint64_t>(row);
#pragma unroll
    for (int i = 0; i < 32 / RPI; ++i) {
        const int r = i * RPI + lane / CH;
        const uint64_t src = __shfl_sync(~0u, mine, r);
        const uint32_t dst = tile + (uint32_t)((c / 8) * kTile * 128 + (32 * warp + r) * 128 + ((c % 8) ^ (r & 7)) * 16);
        cp_async16(dst, src ? reinterpret_cast<const uint4 *>(src) + c : any, src != 0);
    }
}

// Values of new tokens that are not finite become zeros; whether there were any.
template <int D>
__device__ __forceinline__ bool take_out(uint8_t *tile, int from)
{
    constexpr int CH = D / 8, RPI = 32 / CH;
    const int lane = threadIdx.x & 31, warp = threadIdx.x / 32 & 3, c = lane % CH;
    bool any = false;
    for (int i = 0; i < 32 / RPI; ++i) {
        const int r = i * RPI + lane / CH;
        if (32 * warp + r < from)
            continue;
        uint4 *at = reinterpret_cast<uint4 *>(tile + (c / 8) * kTile * 128 + (32 * warp + r) * 128 + ((c % 8) ^ (r & 7)) * 16);
        uint4 v = *at;
        uint32_t *w = &v.x;
        bool here = false;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const uint32_t lo = (w[e] & 0x7F80u) == 0x7F80u ? 0xFFFFu : 0u, hi = (w[e] & 0x7F800000u) == 0x7F800000u ? 0xFFFF0000u : 0u;
            here |= (lo | hi) != 0;
            w[e] &= ~(lo | hi);
        }
        if (here)
            *at = v;
        any |= here;
    }
    return any;
}

template <int D>
__device__ void produce(const AttnParams &p, Smem<D> &sm, Items it)
{
    using S = Smem<D>;
    const int lane = threadIdx.x & 31, warp = threadIdx.x / 32 & 3;
    struct Flight {
        int32_t slot, from, item;  // from: first row among the new tokens' values, kTile: nothing to look at
    } fl[kLag + 1];
    constexpr int kNone = -1, kRows = -2;
#pragma unroll
    for (auto &f : fl)
        f.slot = kNone;
    int c = 0, kt = 0, item = 0;
    const auto land = [&](const Flight &f) {  // what was issued kLag copies ago has arrived
        if (f.slot == kNone)
            return;
        if (f.from < kTile && take_out<D>(sm.ring[f.slot], f.from))
            sm.odd[f.item & 1] = f.item + 1;
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");  // the MMA reads through the async proxy
        __syncwarp();
        if (lane == 0)
            mbar_arrive(smem_u32(f.slot == kRows ? &sm.q_full : &sm.full[f.slot]));
    };
    const auto issued = [&](int slot, int from) {
        asm volatile("cp.async.commit_group;" ::: "memory");
#pragma unroll
        for (int i = 0; i < kLag; ++i)
            fl[i] = fl[i + 1];
        fl[kLag] = Flight{slot, from, item};
        asm volatile("cp.async.wait_group %0;" ::"n"(kLag) : "memory");
        land(fl[0]);
    };
    const auto drain = [&] {
        asm volatile("cp.async.wait_group 0;" ::: "memory");
#pragma unroll
        for (int i = 1; i <= kLag; ++i) {
            land(fl[i]);
            fl[i].slot = kNone;
        }
    };
    bool ok = true;
    do {
        // The rows.  Their buffers are free once the item before has multiplied them all, the second one
        // once its sums are joined.
        drain();  // (the item before ends only with its last copies)
        if (item > 1)
            ok = ok && wait_warp(sm, sm.joined[item & 1], (uint32_t)(item - 2) >> 1 & 1, p, DEP_DEV_TIMEOUT_PRODUCER);
        if (item > 0)
            ok = ok && wait_warp(sm, sm.q_empty, (uint32_t)(item - 1) & 1, p, DEP_DEV_TIMEOUT_PRODUCER);
        if (item > 0 && it.two())
            ok = ok && wait_warp(sm, sm.joined[(item - 1) & 1], (uint32_t)(item - 1) >> 1 & 1, p, DEP_DEV_TIMEOUT_PRODUCER);
        if (!ok)
            break;
        for (int h = 0; h < (it.two() ? 2 : 1); ++h) {
            const int r = kTile * h + 32 * warp + lane, row = it.row0() + r;
            const uint16_t *src = r < it.rows() ? p.q + (it.q.first + row / it.q.G) * p.qs + (it.kv_head * it.q.G + row % it.q.G) * D : nullptr;
            gather<D>(smem_u32(sm.q[h]), src, p.q);
        }
        issued(kRows, kTile);

        const int n = it.t1 - it.t0, own = it.q.own(), end = p.tree ? it.q.len - max(0, it.q.n - kTreeMost) : it.q.len;
        const bool two = it.two();
        const auto load = [&](int t, bool values) {
            const int pos = t * kTile + 32 * warp + lane;
            const int32_t pg = page_of(p, it.s, pos, end);
            const int slot = c % S::kSlots;
            ok = ok && wait_warp(sm, sm.empty[slot], ((uint32_t)(c / S::kSlots) & 1) ^ 1, p, DEP_DEV_TIMEOUT_PRODUCER);
            if (!ok)
                return;
            const int at = pos % p.page;
            const uint16_t *src = nullptr;
            if (pg >= 0)
                src = values ? p.vc + pg * p.vps + at * p.vss + it.kv_head * p.vhs : p.kc + pg * p.kps + at * p.kss + it.kv_head * p.khs;
            if (!values) {
                const uint32_t in = __ballot_sync(~0u, pg >= 0);
                if (lane == 0)
                    sm.masks[kt % kMasks][warp] = in;
                ++kt;
            }
            gather<D>(smem_u32(sm.ring[slot]), src, p.q);
            issued(slot, values && (t + 1) * kTile > own ? max(0, own - t * kTile) : kTile);
            ++c;
        };
        if (two) {
            for (int t = it.t0; ok && t < it.t1; ++t) {
                load(t, false);
                load(t, true);
            }
        } else {
            load(it.t0, false);
            if (n > 1)
                load(it.t0 + 1, false);
            for (int t = it.t0; ok && t < it.t1; ++t) {
                load(t, true);
                if (t + 2 < it.t1)
                    load(t + 2, false);
            }
        }
        ++item;
    } while (ok && it.next(p));
    drain();
}

// ---- multiplying (one thread) -----------------------------------------------------------------

template <int D>
__device__ void multiply(const AttnParams &p, Smem<D> &sm, Items it, uint32_t tmem)
{
    using S = Smem<D>;
    constexpr uint32_t kScores = tc::idesc_bf16_f32(kTile, kTile), kValues = tc::idesc_bf16_f32(kTile, D) | (1u << 16);
    int c = 0, item = 0, k[2] = {0, 0};  // tiles that each group was given
    int sk = 0, sv = 0;  // slots of the first group's keys and values, which the second group shares
    bool ok = true;
    const auto take = [&] {  // the next slot of the ring, once it is full
        const int slot = c % S::kSlots;
        ok = ok && wait(sm, sm.full[slot], (uint32_t)(c / S::kSlots) & 1, p, DEP_DEV_TIMEOUT_MMA);
        ++c;
        return slot;
    };
    const auto scores = [&](int g, int slot, bool two) {
        uint32_t acc = 0;
        tc::mma_steps<D / 16, kTile * 128, kTile * 128>(tmem + g * kTile, tc::desc_sw128(smem_u32(sm.q[two ? g : 0])),
                                                        tc::desc_sw128(smem_u32(sm.ring[slot])), kScores, acc);
        tc::commit(smem_u32(&sm.s_full[g]));
    };
    const auto sums = [&](int g, int slot, bool first) {
        ok = ok && wait(sm, sm.p_full[g], (uint32_t)k[g] & 1, p, DEP_DEV_TIMEOUT_MMA);
        if (!ok)
            return;
        ++k[g];
        tc::fence_after();
        const uint64_t v = desc_values(smem_u32(sm.ring[slot]));
#pragma unroll
        for (int i = 0; i < kTile / 16; ++i)
            mma_bf16_ta(tmem + 2 * kTile + g * D, tmem + g * kTile + 8 * i, v + (uint64_t)(i * 2048 >> 4), kValues, !(first && i == 0));
    };
    const auto release = [&](int slot) { tc::commit(smem_u32(&sm.empty[slot])); };
    do {
        const bool two = it.two();
        const int n[2] = {it.count(0), it.count(1)};
        ok = ok && wait(sm, sm.q_full, (uint32_t)item & 1, p, DEP_DEV_TIMEOUT_MMA);
        if (!ok)
            break;
        tc::fence_after();
        for (int i = -1; ok && i < n[0]; ++i)
            for (int g = 0; ok && g < 2; ++g) {
                if (i >= 0 && i < n[g]) {
                    const int slot_v = two && g == 1 ? sv : take();
                    if (!ok)
                        break;
                    sums(g, slot_v, i == 0);
                    if (!ok)
                        break;
                    sv = slot_v;
                    if (!two || g == 1)
                        release(slot_v);
                    if (i + 1 == n[g])
                        tc::commit(smem_u32(&sm.o_full[g]));
                }
                if (i + 1 < n[g]) {
                    const int slot_k = two && g == 1 ? sk : take();
                    if (!ok)
                        break;
                    tc::fence_after();
                    scores(g, slot_k, two);
                    sk = slot_k;
                    if (!two || g == 1)
                        release(slot_k);
                }
            }
        tc::commit(smem_u32(&sm.q_empty));
        ++item;
    } while (ok && it.next(p));
    if (!ok) {  // what is in flight ends before the tensor memory is given back
        tc::commit(smem_u32(&sm.drained));
        mbar_wait(smem_u32(&sm.drained), 0, kWaitNs);
    }
}

// ---- softmax ----------------------------------------------------------------------------------

template <int D>
__device__ void soften(const AttnParams &p, Smem<D> &sm, Items it, uint32_t tmem, int64_t units, int blocks)
{
    const int g = threadIdx.x / kTile, r = threadIdx.x % kTile, warp = r / 32, lane = r % 32;
    const uint32_t lanes = (uint32_t)(32 * warp) << 16, s_at = tmem + lanes + g * kTile, o_at = tmem + lanes + 2 * kTile + g * D;
    const float c = p.scale * 1.4426950408889634f;  // log2(e)
    int k = 0, kt = 0, item = 0, done = 0, x = 0;  // x: exchanges between the groups
    bool ok = true;
    do {
        const bool two = it.two();
        const int n = it.count(g), at = two ? g * kTile + r : r;
        const bool live = at < it.rows(), warp_live = at - lane < it.rows();
        const int row = it.row0() + at, tok = live ? row / it.q.G : 0, own = it.q.own();
        const int64_t token = it.q.first + tok;
        const uint64_t word = p.tree && live ? p.tree[token] : 0;
        float m = -INFINITY, l = 0.0f;  // m: log2 units
        if (item > 1)  // (a group without tiles does not run ahead)
            ok = wait_warp(sm, sm.joined[item & 1], (uint32_t)(item - 2) >> 1 & 1, p, DEP_DEV_TIMEOUT_CONSUMER);
        for (int i = 0; ok && i < n; ++i, ++k) {
            const int t = it.tile(g, i);
            ok = wait_warp(sm, sm.s_full[g], (uint32_t)k & 1, p, DEP_DEV_TIMEOUT_CONSUMER);
            if (!ok)
                break;
            tc::fence_after();
            if (warp_live) {
                // What the row sees of the tile.
                const uint32_t *in = sm.masks[(kt + (t - it.t0)) % kMasks];
                uint32_t see[4];
                bool all = true;
#pragma unroll
                for (int w = 0; w < 4; ++w) {
                    see[w] = in[w] & seen32(p, own, tok, word, t * kTile + 32 * w);
                    all = all && see[w] == ~0u;
                }
                const bool masked = __any_sync(~0u, !all);
                float top = -INFINITY;
                uint32_t v[32];
#pragma unroll
                for (int w = 0; w < 4; ++w) {
                    tmem_ld32(s_at + 32 * w, v);
                    tc::wait_ld();
                    if (masked) {
#pragma unroll
                        for (int j = 0; j < 32; ++j)
                            top = fmaxf(top, see[w] >> j & 1 ? __uint_as_float(v[j]) : -INFINITY);
                    } else {
#pragma unroll
                        for (int j = 0; j < 32; ++j)
                            top = fmaxf(top, __uint_as_float(v[j]));
                    }
                }
                // The maximum that is taken off moves only where it has risen by 2^8: P stays below 2^8, and
                // O is seldom scaled.
                const float tm = top * c;
                const bool up = tm > m + 8.0f || (m == -INFINITY && tm > -INFINITY);
                if (__any_sync(~0u, up)) {
                    const float f = up ? ex2(m - tm) : 1.0f;
                    if (up)
                        m = tm;
                    l *= f;
                    if (i > 0)  // (the product before is done: this tile's scores came after it)
#pragma unroll
                        for (int w = 0; w < D / 32; ++w) {
                            tmem_ld32(o_at + 32 * w, v);
                            tc::wait_ld();
#pragma unroll
                            for (int j = 0; j < 32; ++j)
                                v[j] = __float_as_uint(__uint_as_float(v[j]) * f);
                            tmem_st32(o_at + 32 * w, v);
                        }
                }
                const float off = m == -INFINITY ? 0.0f : -m;
#pragma unroll
                for (int w = 0; w < 4; ++w) {
                    tmem_ld32(s_at + 32 * w, v);
                    tc::wait_ld();
                    uint32_t pk[16];
                    float add = 0.0f;
#pragma unroll
                    for (int j = 0; j < 32; j += 2) {
                        float a = ex2(fmaf(__uint_as_float(v[j]), c, off)), b = ex2(fmaf(__uint_as_float(v[j + 1]), c, off));
                        if (masked) {
                            a = see[w] >> j & 1 ? a : 0.0f;
                            b = see[w] >> (j + 1) & 1 ? b : 0.0f;
                        }
                        add += a + b;
                        pk[j / 2] = pack16(a, b);
                    }
                    l += add;
                    tmem_st16(s_at + 16 * w, pk);
                }
                tmem_wait_st();
            }
            tc::fence_before();
            __syncwarp();
            if (lane == 0)
                mbar_arrive(smem_u32(&sm.p_full[g]));
        }
        kt += it.t1 - it.t0;
        if (ok && n > 0) {
            ok = wait_warp(sm, sm.o_full[g], (uint32_t)done & 1, p, DEP_DEV_TIMEOUT_EPILOGUE);
            ++done;
            tc::fence_after();
        }
        if (!ok)
            break;
        // Without a second tile of rows the groups' sums are joined: the second group's through shared memory.
        const bool join = !two && it.count(1) > 0;
        float *const scratch = reinterpret_cast<float *>(sm.q[1]);  // [D / 2][kTile]
        float f_own = 1.0f, f_other = 0.0f;
        const bool stores = two || g == 0;
        const bool whole = it.t0 == 0 && it.t1 == it.T;
        const int64_t part = ((int64_t)blockIdx.x * 2 + (it.t0 > 0 ? 0 : 1)) * p.part_rows + at;
        float inv = 1.0f;
        uint16_t *const out = p.o + token * p.os + (it.kv_head * it.q.G + row % it.q.G) * (int64_t)D;
#pragma unroll
        for (int w = 0; w < D / 32; ++w) {
            __syncwarp();
            if (join && w % (D / 64) == 0) {  // half of the channels at once
                if (g == 1) {
                    ok = ok && wait_warp(sm, sm.x_free, ((uint32_t)x & 1) ^ 1, p, DEP_DEV_TIMEOUT_EPILOGUE);
                    if (ok && warp_live) {
                        sm.ml[0][r] = m;
                        sm.ml[1][r] = l;
#pragma unroll
                        for (int u = w; u < w + D / 64; ++u) {
                            uint32_t v[32];
                            tmem_ld32(o_at + 32 * u, v);
                            tc::wait_ld();
#pragma unroll
                            for (int j = 0; j < 32; ++j)
                                scratch[(32 * (u - w) + j) * kTile + r] = __uint_as_float(v[j]);
                        }
                    }
                    __syncwarp();
                    if (lane == 0)
                        mbar_arrive(smem_u32(&sm.x_full));
                } else {
                    ok = ok && wait_warp(sm, sm.x_full, (uint32_t)x & 1, p, DEP_DEV_TIMEOUT_EPILOGUE);
                }
                ++x;
            }
            if (w == 0 && stores) {
                if (join) {
                    const float m1 = sm.ml[0][r], l1 = sm.ml[1][r], top = fmaxf(m, m1);
                    f_own = m == top ? 1.0f : ex2(m - top);
                    f_other = m1 == top ? 1.0f : ex2(m1 - top);
                    l = l * f_own + l1 * f_other;
                    m = top;
                }
                if (whole)
                    inv = l == 0.0f ? 0.0f : 1.0f / l;
            }
            if (!stores)
                continue;
            uint32_t v[32];
            tmem_ld32(o_at + 32 * w, v);
            tc::wait_ld();
            float y[32];
#pragma unroll
            for (int j = 0; j < 32; ++j) {
                y[j] = __uint_as_float(v[j]);
                if (join)
                    y[j] = y[j] * f_own + scratch[(32 * (w % (D / 64)) + j) * kTile + r] * f_other;
                y[j] *= inv;
            }
            if (join && (w + 1) % (D / 64) == 0) {
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(smem_u32(&sm.x_free));
            }
            if (l == 0.0f)
#pragma unroll
                for (int j = 0; j < 32; ++j)
                    y[j] = 0.0f;
            // (both groups' tiles have arrived by now)
            if (*reinterpret_cast<volatile int32_t *>(&sm.odd[item & 1]) == item + 1 && live) {
                // Values that are not finite were left out of the product, which would have given them to every row.
                for (int pos = max(max(own, it.t0 * kTile), 0); pos < min(it.t1 * kTile, it.q.len); ++pos) {
                    const int32_t pg = seen32(p, own, tok, word, pos) & 1 ? page_of(p, it.s, pos, it.q.len) : -1;
                    if (pg < 0)
                        continue;
                    const uint16_t *src = p.vc + pg * p.vps + pos % p.page * p.vss + it.kv_head * p.vhs + 32 * w;
#pragma unroll
                    for (int j = 0; j < 32; ++j)
                        if ((src[j] & 0x7F80u) == 0x7F80u)
                            y[j] += __uint_as_float((uint32_t)src[j] << 16);
                }
            }
            if (!live)
                continue;
            if (whole) {
#pragma unroll
                for (int j = 0; j < 32; j += 8)
                    *reinterpret_cast<uint4 *>(out + 32 * w + j) = make_uint4(pack16(y[j], y[j + 1]), pack16(y[j + 2], y[j + 3]),
                                                                              pack16(y[j + 4], y[j + 5]), pack16(y[j + 6], y[j + 7]));
            } else {
#pragma unroll
                for (int j = 0; j < 32; j += 4)
                    *reinterpret_cast<float4 *>(p.parts + part * D + 32 * w + j) = make_float4(y[j], y[j + 1], y[j + 2], y[j + 3]);
            }
        }
        if (stores && live) {
            if (!whole)
                p.part_ml[part] = make_float2(m, l);
            else if (p.lse)
                p.lse[token * p.Hq + it.kv_head * it.q.G + row % it.q.G] = l == 0.0f ? -INFINITY : (m + log2f(l)) * 0.6931471805599453f;
        }
        if (threadIdx.x == 0 && it.t0 == 0 && it.t1 < it.T) {  // the item goes on in the blocks that follow
            int last = blockIdx.x + 1;
            while (range_begin(units, last + 1, blocks) < it.unit + it.T)
                ++last;
            p.cuts[blockIdx.x] = Cut{last - (int)blockIdx.x + 1, it.s, it.kv_head, it.row0(), it.rows(), {0, 0, 0}};
        }
        tc::fence_before();
        __syncwarp();
        if (lane == 0)
            mbar_arrive(smem_u32(&sm.joined[item & 1]));
        ++item;
    } while (ok && it.next(p));
}

// ---- the kernels ------------------------------------------------------------------------------

template <int D>
__global__ void __launch_bounds__(kThreads, 1) attention_kernel(const AttnParams p)
{
    using S = Smem<D>;
    extern __shared__ uint8_t raw[];
    S &sm = *reinterpret_cast<S *>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~(uintptr_t)1023);
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    griddep_launch_dependents();  // the joining kernel, which waits for this one
    if (warp == kWarps - 1) {
        tc::alloc(smem_u32(&sm.tmem), 512);
        tc::relinquish();
    }
    if (threadIdx.x == 0) {
        for (int i = 0; i < S::kSlots; ++i) {
            mbar_init(smem_u32(&sm.full[i]), kProducers / 32);
            mbar_init(smem_u32(&sm.empty[i]), 1);
        }
        mbar_init(smem_u32(&sm.q_full), kProducers / 32);
        mbar_init(smem_u32(&sm.q_empty), 1);
        mbar_init(smem_u32(&sm.x_full), 4);
        mbar_init(smem_u32(&sm.x_free), 4);
        mbar_init(smem_u32(&sm.drained), 1);
        for (int g = 0; g < 2; ++g) {
            mbar_init(smem_u32(&sm.joined[g]), 8);
            mbar_init(smem_u32(&sm.s_full[g]), 1);
            mbar_init(smem_u32(&sm.p_full[g]), 4);
            mbar_init(smem_u32(&sm.o_full[g]), 1);
        }
        fence_mbar_init();
        sm.dead = 0;
        sm.odd[0] = sm.odd[1] = 0;
        sm.left = 0;
        p.cuts[blockIdx.x].parts = 0;
    }
    // The range.  Every thread adds up the units of its share of the sequences.
    const int per = (p.n_seq + kThreads - 1) / kThreads, s0 = min(p.n_seq, (int)threadIdx.x * per), s1 = min(p.n_seq, s0 + per);
    int64_t mine = 0;
    for (int s = s0; s < s1; ++s) {
        Seq q;
        q.load(p, s);
        mine += q.units(p);
    }
    int64_t before = mine;  // of the warp's lanes up to this one
#pragma unroll
    for (int d = 1; d < 32; d *= 2) {
        const int64_t x = __shfl_up_sync(~0u, before, d);
        before += lane >= d ? x : 0;
    }
    if (lane == 31)
        sm.scan[warp] = before;
    tc::fence_before();
    __syncthreads();
    tc::fence_after();
    int64_t units = 0;
    before -= mine;
    for (int w = 0; w < kWarps; ++w) {
        if (w < warp)
            before += sm.scan[w];
        units += sm.scan[w];
    }
    // At least kLeast tiles a block: fewer are not worth the joining.
    const int blocks = (int)min((int64_t)gridDim.x, max((int64_t)1, units / kLeast));
    const int64_t begin = range_begin(units, blockIdx.x, blocks), end = range_begin(units, blockIdx.x + 1, blocks);
    if ((int)blockIdx.x < blocks && begin < end && begin >= before && begin < before + mine) {
        int s = s0;
        for (;; ++s) {
            Seq q;
            q.load(p, s);
            const int64_t u = q.units(p);
            if (begin < before + u)
                break;
            before += u;
        }
        sm.seq = s;
        sm.unit0 = before;
        sm.left = end - begin;
    }
    __syncthreads();
    const uint32_t tmem = sm.tmem;
    if (sm.left > 0) {
        Items it;
        it.start(p, sm.seq, sm.unit0, begin, sm.left);
        if (warp < 8)
            soften(p, sm, it, tmem, units, blocks);
        else if (warp < 12)
            produce(p, sm, it);
        else if (lane == 0) {
            multiply(p, sm, it, tmem);
        }
    }
    __syncwarp();
    tc::fence_before();
    __syncthreads();
    if (warp == kWarps - 1) {
        tc::fence_after();
        tc::dealloc(tmem, 512);
    }
}

// The parts of the item that begins in block blockIdx.x, joined in the blocks' order; a warp takes a row.
template <int D>
__global__ void __launch_bounds__(256) join_kernel(const AttnParams p)
{
    griddep_wait();
    constexpr int E = D / 32;
    const Cut cut = p.cuts[blockIdx.x];
    if (cut.parts == 0)
        return;
    const int lane = threadIdx.x & 31;
    const int64_t first = seq_start(p, cut.seq);
    const int G = p.Hq / p.Hk;
    for (int r = blockIdx.y * 8 + threadIdx.x / 32; r < cut.rows; r += 8 * gridDim.y) {
        const auto at = [&](int i) { return ((int64_t)(blockIdx.x + i) * 2 + (i == 0 ? 1 : 0)) * p.part_rows + r; };
        float m = -INFINITY;
        for (int i = lane; i < cut.parts; i += 32)
            m = fmaxf(m, p.part_ml[at(i)].x);
#pragma unroll
        for (int d = 16; d; d >>= 1)
            m = fmaxf(m, __shfl_xor_sync(~0u, m, d));
        float l = 0.0f, o[E] = {};
        for (int i = 0; i < cut.parts; ++i) {
            const float2 ml = p.part_ml[at(i)];
            const float f = ml.x == m ? 1.0f : ex2(ml.x - m);
            l = fmaf(ml.y, f, l);
            const float *src = p.parts + at(i) * D + lane * E;
#pragma unroll
            for (int e = 0; e < E; ++e)
                o[e] = fmaf(src[e], f, o[e]);
        }
        const int row = cut.row0 + r, h = cut.kv_head * G + row % G;
        const int64_t token = first + row / G;
        const float inv = l == 0.0f ? 0.0f : 1.0f / l;
        uint32_t w[E / 2];
#pragma unroll
        for (int e = 0; e < E; e += 2)
            w[e / 2] = l == 0.0f ? 0u : pack16(o[e] * inv, o[e + 1] * inv);
        uint32_t *out = reinterpret_cast<uint32_t *>(p.o + token * p.os + (int64_t)h * D) + lane * (E / 2);
#pragma unroll
        for (int e = 0; e < E / 2; ++e)
            out[e] = w[e];
        if (p.lse && lane == 0)
            p.lse[token * p.Hq + h] = l == 0.0f ? -INFINITY : (m + log2f(l)) * 0.6931471805599453f;
    }
}

constexpr int kMostBlocks = 152;  // of a launch: one an SM

// Rows that a part may have: no item has more than all tokens give.
int part_rows(int64_t tokens, int32_t Hq, int32_t Hk) { return (int)std::min<int64_t>(kBlockRows, tokens * (Hq / Hk)); }

// Of the cuts (a multiple of 16 bytes), the parts' m and sums, and the parts; the last on 16 bytes for any number of rows.
int64_t parts_offset(int rows) { return kMostBlocks * (int64_t)(sizeof(Cut) + 2 * rows * sizeof(float2)); }
int64_t workspace_bytes(int rows, int D) { return parts_offset(rows) + kMostBlocks * 2ll * rows * 4 * D; }

cudaError_t device_blocks(int *blocks)
{
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess)
        e = cudaDeviceGetAttribute(blocks, cudaDevAttrMultiProcessorCount, dev);
    return e;
}

template <int D>
cudaError_t attn_launch(AttnParams p, uint8_t *w, cudaStream_t s)
{
    static std::atomic<uint64_t> devices{0};
    cudaError_t e = set_smem_attr(attention_kernel<D>, devices);
    int blocks = 0;
    if (e == cudaSuccess)
        e = device_blocks(&blocks);
    if (e != cudaSuccess)
        return e;
    if (blocks > kMostBlocks)
        blocks = kMostBlocks;
    p.cuts = reinterpret_cast<Cut *>(w);
    p.part_ml = reinterpret_cast<float2 *>(w + kMostBlocks * sizeof(Cut));
    p.parts = reinterpret_cast<float *>(w + parts_offset(p.part_rows));
    static_assert(sizeof(Smem<D>) + 1024 <= kMaxDynamicSmem, "shared memory");
    attention_kernel<D><<<(unsigned)blocks, kThreads, sizeof(Smem<D>) + 1024, s>>>(p);
    e = cudaGetLastError();
    if (e != cudaSuccess)
        return e;
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)blocks, 4);
    cfg.blockDim = dim3(256);
    cfg.stream = s;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, join_kernel<D>, p);
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
        tree{a->tree, 8 * T, 0, a->tree ? 1 : 0}, w{a->workspace, need, 0, need > 0 ? 1 : 0}, st{a->status, 4, 0, a->status ? 1 : 0};
    if (!q.aligned(16) || !o.aligned(16) || !kc.aligned(16) || !vc.aligned(16) || !w.aligned(16) || !st.aligned(4) || !tree.aligned(8) ||
        !lse.aligned(4) || !cu.aligned(4) || !kv.aligned(4) || !table.aligned(4))
        return DEP_ERR_MISALIGNED;
    const Rows ks = kc.span(), vs = vc.span();
    for (const Rows *in : {&q, &cu, &kv, &table, &tree, &ks, &vs})
        if (overlap(o, *in) || overlap(lse, *in) || overlap(w, *in))
            return DEP_ERR_INVALID_ARG;
    if (overlap(o, lse) || overlap(o, w) || overlap(lse, w) || overlap(o, st) || overlap(lse, st) || overlap(w, st))
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
    p.scale = a->scale, p.status = a->status, p.part_rows = part_rows(T, a->Hq, a->Hk);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    uint8_t *const ws = static_cast<uint8_t *>(a->workspace);
    const cudaError_t e = a->D == 128 ? attn_launch<128>(p, ws, s) : attn_launch<64>(p, ws, s);
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
    *bytes = a->tokens == 0 ? 0 : dep::workspace_bytes(dep::part_rows(a->tokens, a->Hq, a->Hk), a->D);
    return DEP_OK;
}

dep_status_t dep_paged_attention(const dep_attention_args_t *args, void *stream)
{
    return dep::attn_entry(args, stream);
}

}  // extern "C"
