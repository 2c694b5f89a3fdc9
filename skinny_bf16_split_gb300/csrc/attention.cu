// attention.cu -- attention of new tokens over a paged cache, on tcgen05.
//
//     o = sum_j p_j v_j / sum_j p_j,  p_j = exp2(c (q . k_j) - m),  c = scale log2(e)
//
// in one pass over the keys and values, with any m: P and the sums are floating point, so m has only to
// keep them in range (see soften()).  P is rounded to BF16, as v is: an MMA takes both operands in one 16-bit
// type, and a second product with what the rounding leaves would be half as much again for the tensor cores, which bound
// the trees.  Errors of at most 2^-8 of each p, of either sign: o is 0.0023 (rms) off where its own rounding makes 0.0017.
// The sum is that of the p before rounding; scores, sums and O are FP32.
//
// Rows.  The n tokens of a sequence and the G = Hq / Hk query heads that share a key and value head are
// the rows of one product: row r is token r / G, head r % G of the G.  A block takes up to 256 of them
// (two tiles of 128, the MMA's M) against tiles of 128 positions: S = Q K^T into tensor memory, a warp
// group for each tile of rows turns its S into P (BF16, in S's own columns, the MMA's A operand from
// tensor memory) and the MMA adds P V to O, which stays in tensor memory.  With 128 rows or fewer the two
// groups take every other tile of positions and the first one joins their sums at the end (both read the same lanes of
// the tensor memory), so that both are at work whatever the number of rows: a tile of M = 128 that holds
// twelve rows of a decode token costs the tensor cores 1024 cycles for the 64 KB that take HBM 2800.
//
// Work.  Every sequence, key and value head and block of rows is an item of ceil(positions seen / 128)
// tiles; the items' tiles, laid end to end with a few tiles' worth for the item itself, are cut into equal
// ranges for one block an SM, so contexts of any lengths fill the GPU evenly.  A block works its range
// out from the lengths on the device.  An item that is cut leaves FP32 parts with their m and sum in the
// workspace; a second kernel joins them in order.
//
// Warps.  Two produce, one keys and one values, each a ring of its own (so neither can be a lap ahead): a tile comes in TMA
// boxes of whole groups of eight slots of a page, or by 16-byte copies where pages have no such groups.  The
// keys' warp also tells the others the items.  Two warps issue MMAs, one for each group; with two tiles of
// rows they take turns.  Values past the end would turn P's zeros into NaN if they are not finite, and
// those of new tokens that some rows do not see likewise: such rows of a tile are looked at on arrival, set to zero,
// and what was not finite is added to the rows that see it at the end.
//
// Bound, with 8 key and value heads of 128 channels, pages of 64 and 96 query heads, of measured rates: one
// token over 131072 positions 94 us (84 % of the copy rate), 64 over 4096 on average, ragged, 183 (87 %): HBM;
// 8 trees of 64 over 16384 positions 310 to 350 us as the clock allows (1.2 to 1.3 PFLOP/s, 62 to 70 % of the
// burst rate; the tensor pipe is active 61 % of the time), a prompt of 8192 tokens 1240 (70 %): the chain of a group's softmax
// (820 cycles a tile alone, 1200 beside the other's) and its products: alone, an MMA of the scores takes 88 cycles instead of
// 64 (both operands from shared memory, 94 bytes a cycle) and one of the values 80, so the 16 of a tile 1350 and their waits
// 100; only the two kinds side by side come to 65.  Two groups in turn make 2900 cycles of that for a pair of tiles, which take
// 3500 to 3950; the rest is not accounted for.  One token over 512 positions 12.7 us: latencies of the lengths, the range, the first
// tile, the softmax, the parts and the joining.  Heads of 64 channels: 58 and 152 us for the first two (68 and 52 % of the copy
// rate), pages that hold no groups of eight slots 205 and 427: not accounted for either.
//
// What was tried and dropped: keys and values by 16-byte copies alone (27 cycles an instruction, 19 B a cycle
// and SM); prefetches into the L2 (8 trees of 64: 322 -> 345 us and more); polls instead of sleeping waits (64 ragged contexts
// 178 -> 279); part of the exponentials on the FMA pipe (337 -> 371, issue slots bound the softmax); the blocks of rows of
// one head side by side over parts of the grid, so that they would read a tile at about the same time (8 trees of 64 took as
// long, and every call a microsecond more to find its range); P handed over in halves, so that its product starts earlier (the
// trees 306 to 317 -> 329: shorter runs of MMAs, a second wait; 64 ragged contexts 179 -> 183); a masked form of the
// straight-line softmax (fetching).
#include <cuda_bf16.h>

#include <math.h>

#include <algorithm>

#include "internal.h"
#include "layer.h"
#include "ptx.cuh"

namespace dep {
namespace {

constexpr int kTreeMost = 64;    // tokens of a sequence that a tree's words name
constexpr int kTile = 128;       // positions of a tile; rows of an MMA
constexpr int kBlockRows = 2 * kTile;  // rows of an item
constexpr int kProducers = 2;    // warps that fetch: one keys, one values
constexpr int kWarps = 12;       // 4 + 4 softmax, 2 producing, 2 issuing MMAs
constexpr int kThreads = 32 * kWarps;
constexpr int kSlotRing = 5 * 32768;  // bytes of keys and values in flight
constexpr int kLanded = 4;  // tiles of values that came in boxes and are looked at: more than are in flight
constexpr int kMasks = 8;   // tiles whose masks are held
constexpr int kAhead = 4;   // items whose descriptions are held
constexpr int kCost = 2;     // tiles' worth of work that an item costs beside its tiles,
constexpr int kCostTwo = 4;  // and one with two tiles of rows
constexpr int kLeast = 1;   // units of a block at least
constexpr uint64_t kWaitNs = 1000000000ull;
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
constexpr float kLift = 12.0f;  // of m over a row's maximum (and zero), log2 units: then a tile's sum is at most one (see soften())
constexpr float kLifted = 0x1p12f;  // 2^kLift
constexpr float kFar = 0x1p28f;  // log2 units; a maximum of that size is held to 16 units at best (see soften())

struct AttnParams {
    const uint16_t *q, *kc, *vc;
    const int32_t *table, *lens, *cu;
    const uint64_t *tree;
    uint16_t *o;
    float *lse;
    int64_t qs, os, kps, kss, khs, vps, vss, vhs, ts;
    int64_t tokens, each, n_pages;  // each: tokens of a sequence where there is no table of starts
    int32_t n_seq, Hq, Hk, G, page, most;  // G = Hq / Hk; most: positions that a row of the table covers
    uint32_t page_mul, page_shift;         // pos / page = pos * page_mul >> page_shift
    float scale;
    int *status;
    int32_t hold;      // a DEP_DEV_* code: waits of that kind are never over (the self-test); else 0
    int32_t part_rows;
    bool wide;         // rows of o start at multiples of 32 bytes
    int32_t box;       // slots of a page in one box of the caches' maps; 0: no maps
    struct Cut *cuts;  // of every block
    float2 *part_ml;   // m and sum of a part's rows: [block][2][part_rows]
    float *parts;      // their channels
};

// What a block leaves for the joining kernel where one of its items goes on in other blocks.
struct Cut {
    int32_t parts;  // of the item; 0: none begins here and goes on
    int32_t kv_head, row0, rows;
    int64_t first;
    int32_t dead;  // a wait of the block gave up
    int32_t pad;
};

// One key and value head of a sequence, up to kBlockRows of its rows, and the tiles [t0, t1) of their T.
struct Item {
    int64_t first;               // the sequence's first token
    int32_t seq, kv_head, row0, rows;
    int32_t t0, t1, T;           // t1 = 0: no more items
    int32_t own, shared, end;    // positions: the first new token's; those before `shared` are seen by all rows, from `end` on by none
    __device__ bool two() const { return rows > kTile; }  // both groups on the same tiles of positions
    __device__ bool whole() const { return t0 == 0 && t1 == T; }
};

struct Dead {
    int32_t here;      // a wait of the block gave up
    int32_t *outside;  // where the joining kernel looks
};

template <int D>
struct Smem {
    static constexpr int kTileBytes = kTile * D * 2;
    static constexpr int kSlots = kSlotRing / kTileBytes, kKeySlots = kSlots / 2;
    // Columns of tensor memory: scores (and P in them) 0 and 128, sums from 256; with 64 channels there is room for P in
    // columns of its own.  Then a group that has every other tile gets its next scores while P is still being multiplied:
    // one token over 131072 positions, 96 heads over 8, 66.0 -> 56.5 us when it came, 64 over 4096 on average 151 -> 146.  Where both
    // groups have the same tiles that order costs more than it gives (8 trees of 64 over 16384 254 -> 285, scores last 260).
    static constexpr bool kApart = D == 64;
    __device__ static constexpr uint32_t p_column(int g) { return kApart ? 2 * kTile + 2 * D + g * (kTile / 2) : g * kTile; }
    uint8_t q[2][kTileBytes];          // tiles of rows
    uint8_t ring[kSlots][kTileBytes];  // a ring of kKeySlots tiles of keys and one of values
    uint64_t full[kSlots], empty[kSlots];
    uint64_t q_full[2], q_empty[2], item_full[kAhead], done[kAhead];
    uint64_t landed[kLanded], turn[2];
    uint64_t s_full[2], p_full[2], p_empty[2], o_full[2], x_full, x_free, drained[2];
    alignas(16) uint32_t masks[kMasks][4];  // positions of a tile that are in the cache
    Item items[kAhead];
    int32_t odd[kAhead];  // 1 + the last item of that place with values of new tokens that are not finite
    float2 ml[kTile];     // the second group's m and sum
    int64_t scan[kWarps];
    int64_t begin, left, unit0;  // this block's range, and the units before its first sequence
    int64_t first;  // its first sequence: as in Seq
    int32_t seq, n, len;
    uint32_t tmem;
    Dead dead;
};

// ---- a sequence, and the items of a range -----------------------------------------------------

__device__ __forceinline__ int64_t seq_start(const AttnParams &p, int s)
{
    if (!p.cu)
        return p.each * s;
    const int64_t t = p.cu[s];
    return t < 0 ? 0 : t > p.tokens ? p.tokens : t;
}

struct Seq {
    int64_t first;  // token
    int32_t n, len, rows, blocks;
    __device__ void load(const AttnParams &p, int s)
    {
        const int32_t l = p.lens[s];
        first = seq_start(p, s);
        n = (int32_t)max(seq_start(p, s + 1) - first, (int64_t)0);
        len = min(max(l, 0), p.most);
        derive(p);
    }
    __device__ void derive(const AttnParams &p)
    {
        rows = n * p.G;
        blocks = (rows + kBlockRows - 1) / kBlockRows;
    }
    // What the rows of block rb see ends before this position.
    __device__ int end(const AttnParams &p, int rb) const
    {
        if (p.tree)
            return len - max(0, n - kTreeMost);
        return len - n + (int)((uint32_t)(min(rows, (rb + 1) * kBlockRows) - 1) / (uint32_t)p.G) + 1;
    }
    __device__ int tiles(const AttnParams &p, int rb) const { return max(1, (end(p, rb) + kTile - 1) / kTile); }
    __device__ int cost(int rb) const { return rows - rb * kBlockRows > kTile ? kCostTwo : kCost; }
    __device__ int64_t head_units(const AttnParams &p) const  // of one key and value head
    {
        if (p.tree)
            return n == 0 ? 0 : (int64_t)(blocks - 1) * (tiles(p, 0) + kCostTwo) + tiles(p, 0) + cost(blocks - 1);
        int64_t u = 0;
        for (int rb = 0; rb < blocks; ++rb)
            u += tiles(p, rb) + cost(rb);
        return u;
    }
};

// a / b, by 32 bits where they do.
__device__ __forceinline__ int64_t divide(int64_t a, int64_t b)
{
    return (a | b) >> 32 == 0 ? (int64_t)((uint32_t)a / (uint32_t)b) : a / b;
}

// Units in equal parts for blocks: block b has those from begin(b) on.
struct Parts {
    int64_t each, more;
    __device__ Parts(int64_t units, int blocks) : each(divide(units, blocks)), more(units - each * blocks) {}
    __device__ int64_t begin(int b) const { return b * each + min((int64_t)b, more); }
};

// The items of a block's range, one after another.  An item has its cost in units before its tiles'.
struct Items {
    Seq q;
    int s, kv_head, rb, T;
    int64_t unit, at, left;  // the item's first unit, where in it the range goes on, units left of the range
    __device__ int cost() const { return q.cost(rb); }
    // Go to unit `begin` of the units from sequence `seq` on, which starts at unit0.
    __device__ void start(const AttnParams &p, const Seq &first, int seq, int64_t unit0, int64_t begin, int64_t count)
    {
        s = seq, left = count, q = first;
        const int64_t head = q.head_units(p), skip = divide(begin - unit0, head);
        kv_head = (int)skip;
        unit = unit0 + skip * head;
        for (rb = 0;; ++rb) {
            T = q.tiles(p, rb);
            if (unit + T + cost() > begin)
                break;
            unit += T + cost();
        }
        at = begin - unit;
    }
    // The next item with tiles in the range, or one with t1 = 0.
    __device__ Item take(const AttnParams &p)
    {
        Item it;
        it.t1 = 0;
        if (left <= 0 || s >= p.n_seq)
            return it;
        const int64_t to = min((int64_t)T + cost(), at + left);
        left -= to - at;
        it.first = q.first, it.seq = s, it.kv_head = kv_head, it.row0 = rb * kBlockRows, it.rows = min(kBlockRows, q.rows - it.row0);
        it.t0 = (int)max(at - cost(), (int64_t)0), it.t1 = (int)max(to - cost(), (int64_t)0), it.T = T;
        it.own = q.len - q.n, it.end = q.end(p, rb);
        it.shared = min(it.end, it.own + (p.tree ? 0 : (int)((uint32_t)it.row0 / (uint32_t)p.G) + 1));
        return it;
    }
    __device__ void next(const AttnParams &p)
    {
        unit += T + cost();
        at = 0;
        if (left <= 0)
            return;
        if (++rb == q.blocks) {
            rb = 0;
            if (++kv_head == p.Hk) {
                kv_head = 0;
                do {
                    if (++s >= p.n_seq)
                        return;
                    q.load(p, s);
                } while (q.n == 0);
            }
        }
        T = q.tiles(p, rb);
    }
};

__device__ __forceinline__ int32_t page_of(const AttnParams &p, int pos) { return (int32_t)((uint64_t)(uint32_t)pos * p.page_mul >> p.page_shift); }

// Bits of the 32 positions from `pos` on that token i of the sequence sees (word: its tree, or null).
__device__ __forceinline__ uint32_t seen32(bool tree, int own, int i, uint64_t word, int pos)
{
    const int at = pos - own;  // of the first position among the new tokens
    if (at <= -32)
        return ~0u;
    if (!tree) {
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
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&v)[16])
{
    asm volatile("tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, "
                 "%14, %15, %16};" ::"r"(taddr),
                 "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]),
                 "r"(v[9]), "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
                 : "memory");
}

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

__device__ __forceinline__ bool mbar_test_wait(uint32_t bar, uint32_t parity)
{
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(bar), "r"(parity)
        : "memory");
    return ok != 0;
}

// Wait for a phase; false if this wait or another one of the block gave up.  (Out of line: fetching code costs.)
__device__ __noinline__ bool wait_long(uint32_t bar, uint32_t parity, volatile Dead *dead, int *status, int code)
{
    const uint64_t t0 = globaltimer_ns();
    while (!mbar_try_wait(bar, parity)) {
        if (dead->here)
            return false;
        if (globaltimer_ns() - t0 > kWaitNs) {
            record_status(status, code);
            *dead->outside = 1;
            dead->here = 1;
            return false;
        }
    }
    return true;
}

template <int D>
__device__ __forceinline__ bool wait(Smem<D> &sm, uint64_t &bar, uint32_t parity, const AttnParams &p, int code)
{
    const uint32_t at = smem_u32(&bar);
    return mbar_try_wait(at, parity) || wait_long(at, parity, &sm.dead, p.status, code);
}

// The same for a warp that waits together, and stays together.
template <int D>
__device__ __forceinline__ bool wait_warp(Smem<D> &sm, uint64_t &bar, uint32_t parity, const AttnParams &p, int code)
{
    return __all_sync(~0u, wait(sm, bar, parity, p, code));
}

template <int D>
__device__ __forceinline__ Item next_item(Smem<D> &sm, int item, const AttnParams &p, int code, bool &ok)
{
    ok = ok && wait_warp(sm, sm.item_full[item % kAhead], (uint32_t)(item / kAhead) & 1, p, code);
    Item it = sm.items[item % kAhead];
    if (!ok)
        it.t1 = 0;
    return it;
}

// Steps of 16 positions in which tile t of the values is multiplied: as far as something is seen.
__device__ __forceinline__ int value_steps(int end, int t) { return min(max((end - t * kTile + 15) / 16, 1), kTile / 16); }

// ---- producing --------------------------------------------------------------------------------

// The first `rows` rows of a swizzled tile, 2 D bytes each, by 16-byte copies of one warp: source(i) is the lane's
// row 32 i + lane (null: zeros).
template <int D, typename Source>
__device__ __forceinline__ void gather(uint32_t tile, int rows, const void *any, Source source)
{
    constexpr int CH = D / 8, RPI = 32 / CH;  // chunks of a row; rows an instruction
    const int lane = threadIdx.x & 31, c = lane % CH;
#pragma unroll 1
    for (int i = 0; 32 * i < rows; ++i) {
        const uint64_t mine = reinterpret_cast<uint64_t>(source(i));
        const uint32_t to = tile + (uint32_t)((c / 8) * kTile * 128 + 32 * i * 128);
#pragma unroll 4
        for (int j = 0; j < CH; ++j) {
            const int r = j * RPI + lane / CH;
            const uint64_t src = __shfl_sync(~0u, mine, r);
            cp_async16(to + (uint32_t)(r * 128 + ((c % 8) ^ (r & 7)) * 16), src ? reinterpret_cast<const uint4 *>(src) + c : any, src != 0);
        }
    }
}

// Rows [from, to) of a swizzled tile of values: those from `end` on become zeros, and of the others what is not
// finite; whether there was any such.
template <int D>
__device__ __forceinline__ bool mend(uint8_t *tile, int from, int end, int to)
{
    constexpr int CH = D / 8, RPI = 32 / CH;
    const int lane = threadIdx.x & 31, c = lane % CH;
    bool any = false;
    constexpr int kAtOnce = 2;
#pragma unroll 1
    for (int i0 = from / RPI * RPI; i0 < to; i0 += kAtOnce * RPI) {
        const auto place = [&](int k) {
            const int r = min(i0 + k * RPI + lane / CH, kTile - 1);
            return reinterpret_cast<uint4 *>(tile + (c / 8) * kTile * 128 + r * 128 + ((c % 8) ^ (r & 7)) * 16);
        };
        uint4 v[kAtOnce];
#pragma unroll
        for (int k = 0; k < kAtOnce; ++k)
            v[k] = *place(k);
#pragma unroll
        for (int k = 0; k < kAtOnce; ++k) {
            const int r = i0 + k * RPI + lane / CH;
            uint32_t *const w = &v[k].x;
            bool here = false;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const uint32_t lo = (w[e] & 0x7F80u) == 0x7F80u ? 0xFFFFu : 0u, hi = (w[e] & 0x7F800000u) == 0x7F800000u ? 0xFFFF0000u : 0u;
                here |= (lo | hi) != 0;
                w[e] &= ~(lo | hi);
            }
            if (r >= end && r < to)
                *place(k) = make_uint4(0, 0, 0, 0);
            else if (here && r >= from && r < to) {
                *place(k) = v[k];
                any = true;
            }
        }
    }
    return any;
}

// One box of a cache's map: p.box slots of a page and head, 64 channels from c0 on.
__device__ __forceinline__ void tma_load_box(uint32_t dst, const CUtensorMap *map, int32_t c0, int32_t slot, int32_t head, int32_t page, uint32_t bar)
{
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(slot), "r"(head), "r"(page), "r"(bar)
        : "memory");
}

// Whatever the others do, all that a producing warp has fetched has landed before the block ends: of each slot of its ring the
// last tile, and the last tiles that would be looked at.  (Out of line: 1501 causal tokens 52.6 -> 51.6 us.)
template <int D>
__device__ __noinline__ void drain(Smem<D> &sm, bool values, int ring, uint32_t lap, int boxed)
{
    using S = Smem<D>;
    for (int slot = values ? S::kKeySlots : 0; slot < (values ? S::kSlots : S::kKeySlots); ++slot)
        mbar_wait(smem_u32(&sm.full[slot]), slot < ring ? lap ^ 1 : lap, kWaitNs);
    for (int b = max(boxed - kLanded, 0); b < boxed; ++b)
        mbar_wait(smem_u32(&sm.landed[b % kLanded]), (uint32_t)(b / kLanded) & 1, kWaitNs);
}

template <int D>
__device__ void produce(const AttnParams &p, Smem<D> &sm, const CUtensorMap &kmap, const CUtensorMap &vmap, const Parts &parts)
{
    using S = Smem<D>;
    constexpr int H = D / 64;
    const int lane = threadIdx.x & 31;
    const bool values = threadIdx.x / 32 != 8;
    // Copies of 16 bytes, and values that have to be looked at, are announced once the next copy has been issued.
    constexpr int kNone = -1, kRows = -2;  // kRows, kRows - 1: the tiles of rows
    struct Flight {
        int32_t slot, item, from, end, to;  // rows of values that have to be looked at, as for mend(); from = to: none
        int32_t box;                        // the number of a tile that came in boxes, or -1
    } flight;
    flight.slot = kNone;
    int ring = values ? S::kKeySlots : 0, item = 0, qc = 0, boxed = 0, kt = 0;
    uint32_t lap = 1;  // of the ring, as the parity that its empty slots have
    bool ok = true;
    // Boxes: lane l issues half l % H of box l / H of a tile.
    const int boxes = p.box ? kTile / p.box : 0, box_row = min(lane / H, boxes - 1) * p.box, half = lane % H;
    const uint32_t box_at = (uint32_t)(half * kTile * 128 + box_row * 128);
    const CUtensorMap *const map = values ? &vmap : &kmap;
    const auto land = [&](bool more = false) {  // more: copies have been issued since
        if (flight.slot == kNone)
            return;
        if (flight.box >= 0)
            ok = wait_warp(sm, sm.landed[flight.box % kLanded], (uint32_t)(flight.box / kLanded) & 1, p, DEP_DEV_TIMEOUT_PRODUCER) && ok;
        else if (more)
            asm volatile("cp.async.wait_group 1;" ::: "memory");
        else
            asm volatile("cp.async.wait_group 0;" ::: "memory");
        if (ok && flight.from < flight.to && mend<D>(sm.ring[flight.slot], flight.from, flight.end, flight.to))
            sm.odd[flight.item % kAhead] = flight.item + 1;
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");  // the MMA reads through the async proxy
        __syncwarp();
        if (lane == 0)
            mbar_arrive(smem_u32(flight.slot <= kRows ? &sm.q_full[kRows - flight.slot] : &sm.full[flight.slot]));
        flight.slot = kNone;
    };
    const auto copied = [&](int slot, int from = 0, int end = 0, int to = 0, int box = -1) {
        asm volatile("cp.async.commit_group;" ::: "memory");
        land(true);
        flight = Flight{slot, item, from, end, to, box};
    };
    // What is waited for may itself wait for copies that have not been announced yet.
    const auto need = [&](uint64_t &bar, uint32_t parity) {
        if (!ok || __all_sync(~0u, mbar_test_wait(smem_u32(&bar), parity)))  // (try_wait would sleep on it)
            return;
        land();
        ok = ok && wait_warp(sm, bar, parity, p, DEP_DEV_TIMEOUT_PRODUCER);
    };
    Items list;
    if (!values)
    {
        Seq q;
        q.first = sm.first, q.n = sm.n, q.len = sm.len;
        q.derive(p);
        list.start(p, q, sm.seq, sm.unit0, sm.begin, sm.left);
    }
    for (;; ++item) {
        if (!values) {  // tells the others
            const Item it = list.take(p);
            if (item >= kAhead)
                need(sm.done[item % kAhead], (uint32_t)(item / kAhead - 1) & 1);
            if (!ok)
                break;  // (others may still be at the item that was there)
            if (lane == 0) {
                sm.items[item % kAhead] = it;
                if (it.t0 == 0 && it.t1 > 0 && it.t1 < it.T) {  // goes on in the blocks that follow
                    int last = blockIdx.x + 1;
                    while (parts.begin(last + 1) < list.unit + it.T + list.cost())
                        ++last;
                    Cut &cut = p.cuts[blockIdx.x];
                    cut.parts = last - (int)blockIdx.x + 1, cut.kv_head = it.kv_head, cut.row0 = it.row0, cut.rows = it.rows;
                    cut.first = it.first;
                }
                mbar_arrive(smem_u32(&sm.item_full[item % kAhead]));
            }
            __syncwarp();
        } else
            need(sm.item_full[item % kAhead], (uint32_t)(item / kAhead) & 1);
        const Item it = sm.items[item % kAhead];
        if (!ok || it.t1 == 0)
            break;
        const bool two = it.two();
        const int n = it.t1 - it.t0;
        const int32_t *const table = p.table + it.seq * p.ts;
        // The page of the lane's box, as the table has it, and the box's slot there; looked up a tile ahead.
        const auto look = [&](int t, int &slot) {
            const int pos = t * kTile + box_row, i = page_of(p, pos);
            slot = pos - i * p.page;
            return boxes && pos < it.end ? table[i] : -1;
        };
        const auto page_at = [&](int pos) {
            const int32_t g = pos < it.end ? table[page_of(p, pos)] : -1;
            return (uint32_t)g < (uint32_t)p.n_pages ? g : -1;
        };
        int next_slot, next_page = look(it.t0, next_slot);
        // Rows: each warp fetches half of a tile, the values' the first one, the keys' its own after its first tile of keys.
        const auto rows = [&] {
            for (int h = 0; h < (two ? 2 : 1); ++h) {
                const int b = (qc + h) & 1, r0 = kTile * h + (values ? 0 : kTile / 2);
                need(sm.q_empty[b], ((uint32_t)((qc + h) >> 1) & 1) ^ 1);
                if (!ok)
                    return;
                gather<D>(smem_u32(sm.q[b]) + (values ? 0 : kTile / 2 * 128), min(kTile / 2, it.rows - r0), p.q, [&](int i) -> const uint16_t * {
                    const int r = r0 + 32 * i + lane;
                    const uint32_t row = it.row0 + r, tok = row / (uint32_t)p.G;
                    return r < it.rows ? p.q + (it.first + tok) * p.qs + (int32_t)(it.kv_head * p.G + (row - tok * p.G)) * D : nullptr;
                });  // (the tile's other rows are nobody's)
                copied(kRows - b);
            }
        };
        if (values)
            rows();
        for (int i = 0; i < n; ++i) {
            const int t = it.t0 + i, slot = ring;
            const int32_t page = (uint32_t)next_page < (uint32_t)p.n_pages ? next_page : -1, in_page = next_slot;
            if (t + 1 < it.t1)
                next_page = look(t + 1, next_slot);
            if (!values) {  // which of the positions are in the cache
                uint32_t *const mask = sm.masks[kt++ % kMasks];
                if (!boxes) {
                    for (int w = 0; w < 4; ++w) {
                        const uint32_t m = __ballot_sync(~0u, page_at(t * kTile + 32 * w + lane) >= 0);
                        if (lane == 0)
                            mask[w] = m;
                    }
                } else if (__all_sync(~0u, page >= 0) && (t + 1) * kTile <= it.end) {
                    if (lane < 4)
                        mask[lane] = ~0u;
                } else {
                    const int here = page < 0 ? 0 : min(max(it.end - (t * kTile + box_row), 0), p.box);
#pragma unroll
                    for (int w = 0; w < 4; ++w) {  // rows [box_row, box_row + here) in those of the word
                        const int lo = min(max(box_row - 32 * w, 0), 32), hi = min(max(box_row + here - 32 * w, 0), 32);
                        const uint32_t m = __reduce_or_sync(~0u, (uint32_t)((1ull << hi) - (1ull << lo)) * (uint32_t)(hi > lo));
                        if (lane == 0)
                            mask[w] = m;
                    }
                }
                __syncwarp();
            }
            // Values past the end have to be zeros, and those that not all rows see finite.
            int from = 0, to = 0, end = 0;
            if (values && (t + 1) * kTile > it.shared) {
                to = 16 * value_steps(it.end, t), end = it.end - t * kTile;
                from = max(0, min(it.shared - t * kTile, to));
            }
            // (everything is worked out by now: a slot that has come free is filled at once)
            need(sm.empty[slot], lap);
            if (!ok)
                break;
            if (++ring == (values ? S::kSlots : S::kKeySlots))
                ring = values ? S::kKeySlots : 0, lap ^= 1;
            if (boxes) {
                const uint32_t bar = smem_u32(from < to ? &sm.landed[boxed % kLanded] : &sm.full[slot]);
                if (lane == 0)
                    mbar_arrive_expect_tx(bar, S::kTileBytes);
                __syncwarp();
                if (lane < boxes * H)  // (a page outside the pool gives zeros)
                    tma_load_box(smem_u32(sm.ring[slot]) + box_at, map, 64 * half, in_page, it.kv_head, page >= 0 ? page : (int32_t)p.n_pages, bar);
                if (from < to)
                    copied(slot, from, end, to, boxed++);
                else
                    land();
            } else {
                const uint16_t *const base = values ? p.vc + it.kv_head * p.vhs : p.kc + it.kv_head * p.khs;
                const int64_t ps = values ? p.vps : p.kps, ss = values ? p.vss : p.kss;
                // (of the values only what the last product reads)
                gather<D>(smem_u32(sm.ring[slot]), values ? 16 * value_steps(it.end, t) : kTile, p.q, [&](int w) -> const uint16_t * {
                    const int pos = t * kTile + 32 * w + lane, g = page_at(pos);
                    return g < 0 ? nullptr : base + g * ps + (pos - page_of(p, pos) * p.page) * ss;
                });
                copied(slot, from, end, to);
            }
            if (!values && i == 0)
                rows();
        }
        qc += two ? 2 : 1;
        if (!values)
            list.next(p);
    }
    land();
    drain(sm, values, ring, lap, boxed);
}

// ---- multiplying (one thread for each group) --------------------------------------------------

template <int D>
__device__ __forceinline__ void multiply_scores(uint32_t s_at, uint64_t rows, uint32_t keys)
{
    constexpr uint32_t kScores = tc::idesc_bf16_f32(kTile, kTile);
    uint32_t acc = 0;
    tc::mma_steps<D / 16, kTile * 128, kTile * 128>(s_at, rows, tc::desc_sw128(keys), kScores, acc);
}

// The first `steps` of a tile's groups of 16 positions.
template <int D>
__device__ __forceinline__ void multiply_values(uint32_t o_at, uint32_t s_at, uint32_t values, int steps, uint32_t acc)
{
    constexpr uint32_t kValues = tc::idesc_bf16_f32(kTile, D) | (1u << 16);
    const uint64_t v = desc_values(values);
    if (steps == kTile / 16) {
#pragma unroll
        for (int j = 0; j < kTile / 16; ++j) {
            mma_bf16_ta(o_at, s_at + 8 * j, v + (uint64_t)(j * 2048 >> 4), kValues, acc);
            acc = 1;
        }
    } else
#pragma unroll 1
        for (int j = 0; j < steps; ++j) {
            mma_bf16_ta(o_at, s_at + 8 * j, v + (uint64_t)(j * 2048 >> 4), kValues, acc);
            acc = 1;
        }
}

template <int D>
__device__ void multiply(const AttnParams &p, Smem<D> &sm, uint32_t tmem, int g)
{
    using S = Smem<D>;
    const uint32_t s_at = tmem + g * kTile, o_at = tmem + 2 * kTile + g * D, p_at = tmem + S::p_column(g), ring = smem_u32(sm.ring[0]);
    const uint32_t empty = smem_u32(&sm.empty[0]);
    bool ok = true;
    int key_slot = 0, value_slot = S::kKeySlots, item = 0, qc = 0;
    uint32_t key_lap = 0, value_lap = 0, k = 0, u = 0;  // of the rings; tiles multiplied; turns taken
    const auto next_keys = [&] {  // the next slot, once it is full
        ok = ok && wait(sm, sm.full[key_slot], key_lap, p, DEP_DEV_TIMEOUT_MMA);
        const int at = key_slot;
        if (++key_slot == S::kKeySlots)
            key_slot = 0, key_lap ^= 1;
        return at;
    };
    const auto next_values = [&] {
        ok = ok && wait(sm, sm.full[value_slot], value_lap, p, DEP_DEV_TIMEOUT_MMA);
        const int at = value_slot;
        if (++value_slot == S::kSlots)
            value_slot = S::kKeySlots, value_lap ^= 1;
        return at;
    };
    // Where both groups have the same tiles they take turns, each with the product of P and the next scores: so
    // one group's products run while the other one softens, instead of both at once and then neither.
    const auto turn = [&] { ok = ok && wait(sm, sm.turn[g], (u & 1) ^ (uint32_t)(g == 0), p, DEP_DEV_TIMEOUT_MMA); };
    const auto pass = [&] {
        mbar_arrive(smem_u32(&sm.turn[g ^ 1]));
        ++u;
    };
    for (;; ++item) {
        ok = ok && wait(sm, sm.item_full[item % kAhead], (uint32_t)(item / kAhead) & 1, p, DEP_DEV_TIMEOUT_MMA);
        const Item &it = sm.items[item % kAhead];
        const int n = it.t1 - it.t0, t0 = it.t0, to = it.end;
        if (!ok || it.t1 == 0)
            break;
        const bool two = it.two();
        // (both tiles of rows, also the other group's: the release below counts on it)
        for (int h = 0; h < (two ? 2 : 1); ++h)
            ok = ok && wait(sm, sm.q_full[(qc + h) & 1], (uint32_t)((qc + h) >> 1) & 1, p, DEP_DEV_TIMEOUT_MMA);
        // The tiles of rows are free for the next item with this group's last scores.
        const auto done_with_rows = [&] {
            for (int h = 0; h < (two ? 2 : 1); ++h)
                tc::commit(smem_u32(&sm.q_empty[(qc + h) & 1]));
        };
        const uint64_t rows = tc::desc_sw128(smem_u32(sm.q[two ? (qc + g) & 1 : qc & 1]));
        if (two) {
            int keys = next_keys();
            turn();
            if (!ok)
                break;
            tc::fence_after();
            multiply_scores<D>(s_at, rows, ring + keys * S::kTileBytes);
            pass();
            tc::commit(smem_u32(&sm.s_full[g]));
            tc::commit(empty + 8 * keys);
            if (n == 1)
                done_with_rows();
            for (int t = 0; t < n; ++t) {
                const int values = next_values();
                if (t + 1 < n)
                    keys = next_keys();
                const uint32_t v_at = ring + values * S::kTileBytes, k_at = ring + keys * S::kTileBytes;
                const int steps = value_steps(to, t0 + t);
                ok = ok && wait(sm, sm.p_full[g], k & 1, p, DEP_DEV_TIMEOUT_MMA);
                ++k;
                turn();
                if (!ok)
                    break;
                tc::fence_after();
                multiply_values<D>(o_at, p_at, v_at, steps, t > 0);
                if (t + 1 < n) {
                    multiply_scores<D>(s_at, rows, k_at);
                    pass();
                    tc::commit(smem_u32(&sm.s_full[g]));
                    tc::commit(empty + 8 * keys);
                    if (t + 2 == n)
                        done_with_rows();
                } else {
                    pass();
                    tc::commit(smem_u32(&sm.o_full[g]));
                }
                tc::commit(empty + 8 * values);
            }
        } else {
            // Every other tile: two tiles' keys first, then a tile's values and the keys of the one after the next (these
            // first, where P has columns of its own).
            const int last = n - 1 - ((n - 1 - g) & 1);  // this group's last tile
            const auto scores = [&](int t) {
                const int at = next_keys();
                if (!ok)
                    return;
                if ((t & 1) != g) {
                    mbar_arrive(empty + 8 * at);  // the other group's
                    return;
                }
                tc::fence_after();
                multiply_scores<D>(s_at, rows, ring + at * S::kTileBytes);
                tc::commit(smem_u32(&sm.s_full[g]));
                tc::commit(empty + 8 * at);
                if (t == last)
                    done_with_rows();
            };
            if (last < 0)
                done_with_rows();
            for (int t = -2; ok && t < n; ++t) {
                if (t >= 0) {
                    const int at = next_values();
                    if (ok && (t & 1) != g)
                        mbar_arrive(empty + 8 * at);
                    else if (ok) {
                        ok = wait(sm, sm.p_full[g], k & 1, p, DEP_DEV_TIMEOUT_MMA);
                        if (!ok)
                            break;
                        ++k;
                        if (S::kApart && t + 2 < n)
                            scores(t + 2);
                        if (!ok)
                            break;
                        tc::fence_after();
                        multiply_values<D>(o_at, p_at, ring + at * S::kTileBytes, value_steps(to, t0 + t), t > 1);
                        if (S::kApart)
                            tc::commit(smem_u32(&sm.p_empty[g]));
                        if (t == last)
                            tc::commit(smem_u32(&sm.o_full[g]));
                        tc::commit(empty + 8 * at);
                        if (S::kApart)
                            continue;
                    }
                }
                if (ok && t + 2 < n)
                    scores(t + 2);
            }
        }
        qc += two ? 2 : 1;
    }
    // What is in flight ends before the tensor memory is given back, also where nobody has waited for it.
    tc::commit(smem_u32(&sm.drained[g]));
    mbar_wait(smem_u32(&sm.drained[g]), 0, kWaitNs);
}

// ---- softmax ----------------------------------------------------------------------------------

__device__ __forceinline__ uint64_t both(float a, float b)
{
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ void apart(uint64_t r, float &a, float &b) { asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(r)); }
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c)
{
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b)
{
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}

// p = exp2(c s + off) of the row's scores of a tile in BF16 pairs; their sum.
__device__ __forceinline__ float tile_exp(uint32_t s_at, float c, float off, uint32_t (&pk)[2][32])
{
    const uint64_t c2 = both(c, c), off2 = both(off, off);
    uint64_t s2[2] = {0, 0};
    uint32_t v[2][16];
    tc::ld16(s_at, v[0]);
#pragma unroll
    for (int w = 0; w < kTile / 16; ++w) {
        tc::wait_ld();
        if (w + 1 < kTile / 16)
            tc::ld16(s_at + 16 * (w + 1), v[(w + 1) & 1]);
#pragma unroll
        for (int j = 0; j < 16; j += 2) {
            float x, y;
            apart(fma2(both(__uint_as_float(v[w & 1][j]), __uint_as_float(v[w & 1][j + 1])), c2, off2), x, y);
            x = ex2(x), y = ex2(y);
            s2[j / 2 & 1] = add2(s2[j / 2 & 1], both(x, y));
            pk[w / 4][8 * (w & 3) + j / 2] = pack16(x, y);
        }
    }
    float x, y;
    apart(add2(s2[0], s2[1]), x, y);
    return x + y;
}

// 32 bytes at a multiple of 32.
__device__ __forceinline__ void store32(void *to, const uint32_t (&v)[8])
{
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(to), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]),
                 "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
                 : "memory");
}

// The logarithm of the sum; m's lift goes into l again, where it is exact: sums of about one keep their precision.  (Out of line, with
// 64 channels and 64 ragged contexts, 159 -> 152 us.)
__device__ __noinline__ float log_sum(float m, float l) { return (m - kLift + log2f(l * kLifted)) * kLn2; }

// Adds the values of new tokens that are not finite, which were left out of the product (it would have
// given them to every row), to the channels of a row that sees them.  FP32 or BF16 in `row`.
template <int D>
__device__ __noinline__ void add_odd(const AttnParams &p, const Item &it, int tok, uint64_t word, uint16_t *out, float *part)
{
    for (int pos = max(max(it.shared, it.t0 * kTile), 0); pos < min(it.t1 * kTile, it.end); ++pos) {
        if (!(seen32(p.tree != nullptr, it.own, tok, word, pos) & 1))
            continue;
        const int32_t pi = page_of(p, pos), pg = p.table[it.seq * p.ts + pi];
        if (pg < 0 || pg >= p.n_pages)
            continue;
        const uint16_t *src = p.vc + pg * p.vps + (pos - pi * p.page) * p.vss + it.kv_head * p.vhs;
        for (int d = 0; d < D; ++d) {
            const float v = __uint_as_float((uint32_t)src[d] << 16);
            if (isfinite(v))
                continue;
            if (part)
                part[d] += v;
            else
                out[d] = __bfloat16_as_ushort(__float2bfloat16_rn(__uint_as_float((uint32_t)out[d] << 16) + v));
        }
    }
}

template <int D>
__device__ void soften(const AttnParams &p, Smem<D> &sm, uint32_t tmem)
{
    const int g = threadIdx.x / kTile, r = threadIdx.x % kTile, lane = r % 32;
    const uint32_t lanes = (uint32_t)(r - lane) << 16, s_at = tmem + lanes + g * kTile, o_at = tmem + lanes + 2 * kTile + g * D;
    const float c = p.scale * kLog2e;
    const bool tree = p.tree != nullptr;
    int kt = 0, item = 0;
    uint32_t k = 0, e = 0, items = 0, x = 0;  // tiles; those with P of its own; items with tiles; exchanges between the groups
    bool ok = true, lent = false;      // lent: the first group may still read this one's sums
    for (;; ++item) {
        const Item it = next_item(sm, item, p, DEP_DEV_TIMEOUT_CONSUMER, ok);
        if (it.t1 == 0)
            break;
        const bool two = it.two(), apart = Smem<D>::kApart && !two;
        const uint32_t p_at = tmem + lanes + Smem<D>::p_column(g);
        const int at = two ? g * kTile + r : r;
        const bool live = at < it.rows, warp_live = at - lane < it.rows;
        const uint32_t row = it.row0 + at;
        const int tok = live ? (int)(row / (uint32_t)p.G) : 0, head = it.kv_head * p.G + (int)(row - tok * p.G);
        const int64_t token = it.first + tok;
        const uint64_t word = tree && live ? p.tree[token] : 0;
        const int clear = it.own + (tree ? 0 : __shfl_sync(~0u, tok, 0) + 1);  // all positions before it are seen by all of the warp's rows
        float m = kLift, l = 0.0f;  // m: log2 units
        int t = it.t0 + (two ? 0 : g);
        const bool some = t < it.t1;
        for (bool first = true; t < it.t1; t += two ? 1 : 2, first = false, ++k, e += apart) {
            ok = ok && wait_warp(sm, sm.s_full[g], k & 1, p, DEP_DEV_TIMEOUT_CONSUMER);
            if (!ok)
                break;
            tc::fence_after();
            // P's own columns are free, and O is settled, once the product before is done (elsewhere that came before these
            // scores).
            const auto last_product = [&] {
                if (apart && e > 0) {
                    if (!wait_warp(sm, sm.p_empty[g], (e - 1) & 1, p, DEP_DEV_TIMEOUT_CONSUMER))
                        ok = false;
                    tc::fence_after();
                }
            };
            if (warp_live) {
                const uint4 in = *reinterpret_cast<const uint4 *>(sm.masks[(kt + (t - it.t0)) % kMasks]);
                // P and its sum keep their precision at any size, so what is taken off, m, is the same for all rows to begin with
                // and moves only where a tile's sum would pass one, or all that was seen stays below 2^-40: then O has seldom
                // to be scaled, and one pass over the scores does.  The sum (in which a NaN shows as well) tells; with another m
                // the tile is taken anew.  (No p is more than one, as with the maximum itself, so O leaves FP32's range for no
                // values for which it would not then.)
                const bool masked = (t + 1) * kTile > clear || (in.x & in.y & in.z & in.w) != ~0u;
                bool wrong = masked, anew = masked;
                float sum = 0.0f;
                if (!masked) {
                    uint32_t pk[2][32];
                    sum = tile_exp(s_at, c, -m, pk);
                    last_product();
                    wrong = live && !(sum <= 1.0f && l + sum >= 0x1p-40f && fabsf(m) < kFar);
                    if (!__any_sync(~0u, wrong)) {
                        l += sum;
                        tmem_st32(p_at, pk[0]);
                        tmem_st32(p_at + 32, pk[1]);
                    } else
                        anew = true;
                }
                if (anew) {  // with what the row sees; rolled up, since it is seldom run: its fetching costs more than its running
                    if (masked)
                        last_product();
                    const uint32_t *mask = sm.masks[(kt + (t - it.t0)) % kMasks];
                    float top = -INFINITY;
#pragma unroll 1
                    for (int w = 0; w < 4; ++w) {
                        uint32_t v[32];
                        tmem_ld32(s_at + 32 * w, v);
                        const uint32_t see = mask[w] & seen32(tree, it.own, tok, word, t * kTile + 32 * w);
                        tc::wait_ld();
#pragma unroll
                        for (int j = 0; j < 32; ++j)
                            top = fmaxf(top, see >> j & 1 ? __uint_as_float(v[j]) : -INFINITY);
                    }
                    const float tm = __fmul_rn(top, c);  // (nothing fused: as a far row's products are below)
                    // (what a row does goes by its own scores: where only others were wrong it comes to the same P again)
                    const bool fresh = l == 0.0f, up = live && wrong && (tm > m - (kLift - 5.0f) || (fresh && tm > -INFINITY));
                    if (__any_sync(~0u, up)) {
                        const float to = !up ? m : fabsf(tm) < kFar ? tm + kLift : tm, f = fresh ? 0.0f : ex2(m - to);
                        m = to;
                        l *= f;
                        if (!first)  // (the product before is done: this tile's scores came after it)
#pragma unroll 1
                            for (int w = 0; w < D / 16; ++w) {
                                uint32_t v[16];
                                tc::ld16(o_at + 16 * w, v);
                                tc::wait_ld();
#pragma unroll
                                for (int j = 0; j < 16; ++j)
                                    v[j] = __float_as_uint(__uint_as_float(v[j]) * f);
                                tmem_st16(o_at + 16 * w, v);
                            }
                    }
                    // p = exp2(c s - m), rounded after the difference alone, is exact in whatever m is, and in range while m is
                    // the row's maximum to a few units.  From 2^28 on FP32 rounds the maximum by eight units and more, in the end
                    // by all that an exponential takes; there c s is rounded first, as the maximum was, and its own p is 1.
                    const float off = -m;
                    const bool far = fabsf(m) >= kFar;
                    const float c1 = far ? 1.0f : c;
                    if (__any_sync(~0u, far)) {
#pragma unroll 1
                        for (int w = 0; w < kTile / 16; ++w) {
                            uint32_t v[16];
                            tc::ld16(s_at + 16 * w, v);
                            tc::wait_ld();
#pragma unroll
                            for (int j = 0; j < 16; ++j)
                                v[j] = __float_as_uint(__fmul_rn(__uint_as_float(v[j]), far ? c : 1.0f));
                            tmem_st16(s_at + 16 * w, v);
                        }
                        tmem_wait_st();
                    }
                    float again = 0.0f;
#pragma unroll 1
                    for (int w = 0; w < 4; ++w) {  // (P's columns lie in those of scores already read)
                        uint32_t v[32], pk[16];
                        tmem_ld32(s_at + 32 * w, v);
                        const uint32_t see = mask[w] & seen32(tree, it.own, tok, word, t * kTile + 32 * w);
                        tc::wait_ld();
#pragma unroll
                        for (int j = 0; j < 32; j += 2) {
                            float a = ex2(fmaf(__uint_as_float(v[j]), c1, off)), b = ex2(fmaf(__uint_as_float(v[j + 1]), c1, off));
                            a = see >> j & 1 ? a : 0.0f;
                            b = see >> (j + 1) & 1 ? b : 0.0f;
                            again += a + b;
                            pk[j / 2] = pack16(a, b);
                        }
                        tmem_st16(p_at + 16 * w, pk);
                    }
                    l += wrong ? again : sum;
                }
                tmem_wait_st();
            }
            if (lent) {
                ok = ok && wait_warp(sm, sm.x_free, (x - 1) & 1, p, DEP_DEV_TIMEOUT_EPILOGUE);
                lent = false;
            }
            tc::fence_before();
            __syncwarp();
            if (lane == 0)
                mbar_arrive(smem_u32(&sm.p_full[g]));
        }
        if (l == 0.0f)
            m = -INFINITY;  // nothing seen
        kt += it.t1 - it.t0;
        if (some) {
            ok = ok && wait_warp(sm, sm.o_full[g], items & 1, p, DEP_DEV_TIMEOUT_EPILOGUE);
            if (apart)  // (a warp without rows has not waited for the products: the next item's wait is for the phase after this)
                ok = ok && wait_warp(sm, sm.p_empty[g], (e - 1) & 1, p, DEP_DEV_TIMEOUT_EPILOGUE);
            ++items;
            tc::fence_after();
        }
        // Without a second tile of rows the first group joins the groups' sums: a warp reads the second group's in its
        // own lanes of the tensor memory.
        const bool join = !two && it.t1 - it.t0 > 1;
        float f_own = 1.0f, f_other = 0.0f;
        if (join && ok) {
            if (g == 1) {
                if (lent)
                    ok = wait_warp(sm, sm.x_free, (x - 1) & 1, p, DEP_DEV_TIMEOUT_EPILOGUE);
                sm.ml[r] = make_float2(m, l);
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(smem_u32(&sm.x_full));
                lent = true;
            } else {
                ok = wait_warp(sm, sm.x_full, x & 1, p, DEP_DEV_TIMEOUT_EPILOGUE);
                tc::fence_after();
                const float2 other = sm.ml[r];
                const float top = fmaxf(m, other.x);
                f_own = m == top ? 1.0f : ex2(m - top);
                f_other = other.x == top ? 1.0f : ex2(other.x - top);
                l = l * f_own + other.y * f_other;
                m = top;
            }
            ++x;
        }
        if (!ok)
            break;
        if (two || g == 0) {
            const bool whole = it.whole();
            const int64_t part = ((int64_t)blockIdx.x * 2 + (it.t0 > 0 ? 0 : 1)) * p.part_rows + at;
            uint16_t *const out = p.o + token * p.os + (int64_t)head * D;
            float *const rest = p.parts + part * D;
            const float inv = l == 0.0f ? 0.0f : whole ? 1.0f / l : 1.0f;
            f_own *= inv;
            f_other *= inv;
            if (warp_live)
#pragma unroll 1
                for (int w = 0; w < D / 16; ++w) {
                    uint32_t v[16], u[16];
                    __syncwarp();
                    tc::ld16(o_at + 16 * w, v);
                    if (join)
                        tc::ld16(o_at + D + 16 * w, u);
                    tc::wait_ld();
                    float y[16];
#pragma unroll
                    for (int j = 0; j < 16; ++j) {
                        y[j] = __uint_as_float(v[j]) * f_own;
                        if (join)
                            y[j] = fmaf(__uint_as_float(u[j]), f_other, y[j]);
                        if (l == 0.0f)
                            y[j] = 0.0f;
                    }
                    if (!live)
                        continue;
                    if (whole) {
                        uint32_t b[8];
#pragma unroll
                        for (int j = 0; j < 8; ++j)
                            b[j] = pack16(y[2 * j], y[2 * j + 1]);
                        if (p.wide)
                            store32(out + 16 * w, b);
                        else {
                            *reinterpret_cast<uint4 *>(out + 16 * w) = make_uint4(b[0], b[1], b[2], b[3]);
                            *reinterpret_cast<uint4 *>(out + 16 * w + 8) = make_uint4(b[4], b[5], b[6], b[7]);
                        }
                    } else {
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            uint32_t b[8];
#pragma unroll
                            for (int j = 0; j < 8; ++j)
                                b[j] = __float_as_uint(y[8 * h + j]);
                            store32(rest + 16 * w + 8 * h, b);
                        }
                    }
                }
            if (join) {
                tc::fence_before();
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(smem_u32(&sm.x_free));
            }
            if (live) {
                // (a row whose scores are all minus infinity has zeros, whatever the values are; of parts the joining sees to it)
                if ((l != 0.0f || !whole) && *reinterpret_cast<volatile int32_t *>(&sm.odd[item % kAhead]) == item + 1)
                    add_odd<D>(p, it, tok, word, out, whole ? nullptr : rest);
                if (!whole)
                    p.part_ml[part] = make_float2(m, l);
                else if (p.lse)
                    p.lse[token * p.Hq + head] = l == 0.0f ? -INFINITY : log_sum(m, l);
            }
        }
        tc::fence_before();
        __syncwarp();
        if (lane == 0)
            mbar_arrive(smem_u32(&sm.done[item % kAhead]));
    }
}

// ---- the kernels ------------------------------------------------------------------------------

template <int D>
__global__ void __launch_bounds__(kThreads, 1) attention_kernel(const __grid_constant__ AttnParams p, const __grid_constant__ CUtensorMap kmap,
                                                               const __grid_constant__ CUtensorMap vmap)
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
            mbar_init(smem_u32(&sm.full[i]), 1);
            mbar_init(smem_u32(&sm.empty[i]), 2 + (p.hold == DEP_DEV_TIMEOUT_PRODUCER));  // (one that never arrives)
        }
        for (int i = 0; i < kAhead; ++i) {
            mbar_init(smem_u32(&sm.item_full[i]), 1);
            mbar_init(smem_u32(&sm.done[i]), 8);
            sm.odd[i] = 0;
        }
        for (int g = 0; g < 2; ++g) {
            mbar_init(smem_u32(&sm.q_full[g]), kProducers);
            mbar_init(smem_u32(&sm.q_empty[g]), 2);
            mbar_init(smem_u32(&sm.s_full[g]), 1 + (p.hold == DEP_DEV_TIMEOUT_CONSUMER));
            mbar_init(smem_u32(&sm.p_full[g]), 4 + (p.hold == DEP_DEV_TIMEOUT_MMA));
            mbar_init(smem_u32(&sm.p_empty[g]), 1);
            mbar_init(smem_u32(&sm.o_full[g]), 1 + (p.hold == DEP_DEV_TIMEOUT_EPILOGUE));
            mbar_init(smem_u32(&sm.drained[g]), 1);
            mbar_init(smem_u32(&sm.turn[g]), 1);
        }
        for (int i = 0; i < kLanded; ++i)
            mbar_init(smem_u32(&sm.landed[i]), 1);
        mbar_init(smem_u32(&sm.x_full), 4);
        mbar_init(smem_u32(&sm.x_free), 4);
        fence_mbar_init();
        sm.dead = Dead{0, &p.cuts[blockIdx.x].dead};
        sm.left = 0;
    }
    griddep_wait();  // what comes before may write the inputs, and read the workspace
    if (threadIdx.x == 0)
        p.cuts[blockIdx.x].parts = p.cuts[blockIdx.x].dead = 0;
    // The range.  Every thread adds up the units of its share of the sequences.
    const int per = (p.n_seq + kThreads - 1) / kThreads, s0 = min(p.n_seq, (int)threadIdx.x * per), s1 = min(p.n_seq, s0 + per);
    int64_t mine = 0;
    Seq q;
#pragma unroll 1
    for (int s = s0; s < s1; ++s) {
        q.load(p, s);
        mine += q.head_units(p) * p.Hk;
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
        const int64_t x = sm.scan[w];
        before += w < warp ? x : 0;
        units += x;
    }
    const int blocks = (int)min((int64_t)gridDim.x, max((int64_t)1, divide(units, kLeast)));
    const Parts parts(units, blocks);
    const int64_t begin = parts.begin(blockIdx.x), end = parts.begin(blockIdx.x + 1);
    if ((int)blockIdx.x < blocks && begin < end && begin >= before && begin < before + mine) {
        int s = s0;
        if (s1 - s0 > 1)  // (else q is still the sequence)
#pragma unroll 1
            for (;; ++s) {
                q.load(p, s);
                const int64_t u = q.head_units(p) * p.Hk;
                if (begin < before + u)
                    break;
                before += u;
            }
        sm.seq = s, sm.first = q.first, sm.n = q.n, sm.len = q.len;
        sm.unit0 = before;
        sm.begin = begin;
        sm.left = end - begin;
    }
    __syncthreads();
    const uint32_t tmem = sm.tmem;
    if (sm.left > 0) {
        if (warp < 8)
            soften(p, sm, tmem);
        else if (warp < 8 + kProducers)
            produce(p, sm, kmap, vmap, parts);
        else if (lane == 0)
            multiply(p, sm, tmem, warp - 8 - kProducers);
    }
    __syncwarp();
    tc::fence_before();
    __syncthreads();
    if (warp == kWarps - 1) {
        tc::fence_after();
        tc::dealloc(tmem, 512);
    }
}

// NaN to the rows of all sequences: a block that gave up does not say which of its own it has done.  Rows that are complete may be
// joined at the same time and stay.
template <int D>
__device__ __noinline__ void spoil(const AttnParams &p)
{
    const int lane = threadIdx.x & 31, warp = blockIdx.y * 8 + threadIdx.x / 32, warps = gridDim.y * 8;
    for (int64_t s = warp; s < p.n_seq; s += warps) {
        const int64_t first = seq_start(p, (int)s), last = seq_start(p, (int)s + 1);
        for (int64_t t = first; t < last; ++t) {
            uint4 *const row = reinterpret_cast<uint4 *>(p.o + t * p.os);
            for (int i = lane; i < p.Hq * (D / 8); i += 32)
                row[i] = make_uint4(0x7FFF7FFFu, 0x7FFF7FFFu, 0x7FFF7FFFu, 0x7FFF7FFFu);
            for (int h = lane; p.lse && h < p.Hq; h += 32)
                p.lse[t * p.Hq + h] = __uint_as_float(0x7FFFFFFFu);
        }
    }
}

// The parts of the item that begins in block blockIdx.x, joined in the blocks' order; a warp takes a row.  What it costs is the
// fetching of its code, it seems, so that is kept short (loops unrolled by more, 64-bit indexes: one token over 512 positions 13.0 -> 13.6 us,
// with 64 channels over 131072 58.4 -> 60.8).
template <int D>
__global__ void __launch_bounds__(256) join_kernel(const AttnParams p)
{
    griddep_launch_dependents();
    griddep_wait();
    constexpr int E = D / 32;
    const Cut cut = p.cuts[blockIdx.x];
    const int lane = threadIdx.x & 31, r = blockIdx.y * 8 + threadIdx.x / 32;
    if (cut.dead)
        return spoil<D>(p);
    if (cut.parts == 0 || r >= cut.rows)
        return;
    const auto at = [&](int i) { return (int)((blockIdx.x + i) * 2 + (i == 0 ? 1 : 0)) * p.part_rows + r; };
    // Lane j: the j-th of 32 parts at once.
    float m = -INFINITY;
    bool lost = false;  // a part that is not complete
#pragma unroll 1
    for (int i = lane; i < cut.parts; i += 32) {
        m = fmaxf(m, p.part_ml[at(i)].x);
        lost |= p.cuts[blockIdx.x + i].dead != 0;
    }
#pragma unroll
    for (int d = 16; d; d >>= 1)
        m = fmaxf(m, __shfl_xor_sync(~0u, m, d));
    float l = lost ? __uint_as_float(0x7FFFFFFFu) : 0.0f, o[E] = {};
#pragma unroll 1
    for (int i0 = 0; i0 < cut.parts; i0 += 32) {
        float f = 0.0f;
        if (i0 + lane < cut.parts) {
            const float2 ml = p.part_ml[at(i0 + lane)];
            f = ml.x == m ? 1.0f : ex2(ml.x - m);
            l = fmaf(ml.y, f, l);
        }
        const int n = min(32, cut.parts - i0);
#pragma unroll 2
        for (int i = 0; i < n; ++i) {
            const float w = __shfl_sync(~0u, f, i);
            const float *src = p.parts + at(i0 + i) * D + lane * E;
            float v[E];
            if (E == 4)
                *reinterpret_cast<float4 *>(v) = *reinterpret_cast<const float4 *>(src);
            else
                *reinterpret_cast<float2 *>(v) = *reinterpret_cast<const float2 *>(src);
#pragma unroll
            for (int e = 0; e < E; ++e)
                o[e] = fmaf(v[e], w, o[e]);
        }
    }
#pragma unroll
    for (int d = 16; d; d >>= 1)
        l += __shfl_xor_sync(~0u, l, d);
    const uint32_t row = cut.row0 + r, tok = row / (uint32_t)p.G;
    const int h = cut.kv_head * p.G + (int)(row - tok * p.G);
    const int64_t token = cut.first + tok;
    const float inv = l == 0.0f ? 0.0f : 1.0f / l;
    uint32_t w[E / 2];
#pragma unroll
    for (int e = 0; e < E; e += 2)
        w[e / 2] = l == 0.0f ? 0u : pack16(o[e] * inv, o[e + 1] * inv);
    uint32_t *out = reinterpret_cast<uint32_t *>(p.o + token * p.os + (int64_t)h * D) + lane * (E / 2);
    if (E == 4)
        *reinterpret_cast<uint2 *>(out) = make_uint2(w[0], w[E / 2 - 1]);
    else
        out[0] = w[0];
    if (p.lse && lane == 0)
        p.lse[token * p.Hq + h] = l == 0.0f ? -INFINITY : log_sum(m, l);
}

constexpr int kMostBlocks = 152;  // of a launch: one an SM

// Rows that a part may have: no item has more than all tokens give.
int part_rows(int64_t tokens, int32_t Hq, int32_t Hk) { return (int)std::min<int64_t>(kBlockRows, std::min<int64_t>(tokens, kBlockRows) * (Hq / Hk)); }

// Of the cuts, the parts' m and sums, and the parts, whole lines of 128 bytes each (a row of a part over one line more: one token
// over 131072 positions 94.1 -> 94.9 us).
constexpr int64_t kCutBytes = kMostBlocks * (int64_t)sizeof(Cut);
static_assert(kCutBytes % 128 == 0 && kMostBlocks * 2 * sizeof(float2) % 128 == 0, "lines");
int64_t parts_offset(int rows) { return kCutBytes + kMostBlocks * 2ll * rows * (int64_t)sizeof(float2); }
int64_t workspace_bytes(int rows, int D) { return parts_offset(rows) + kMostBlocks * 2ll * rows * 4 * D + 128; }

template <int D>
cudaError_t attn_launch(AttnParams p, uint8_t *w, const CUtensorMap &kmap, const CUtensorMap &vmap, cudaStream_t s)
{
    static_assert(sizeof(Smem<D>) + 1024 <= kMaxDynamicSmem, "shared memory");
    static std::atomic<uint64_t> devices{0};
    cudaError_t e = set_smem_attr(attention_kernel<D>, devices);
    int dev = 0, blocks = 0;
    if (e == cudaSuccess)
        e = cudaGetDevice(&dev);
    if (e == cudaSuccess)
        e = cudaDeviceGetAttribute(&blocks, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess)
        return e;
    blocks = std::min(blocks, kMostBlocks);
    w = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(w) + 127) & ~(uintptr_t)127);
    p.cuts = reinterpret_cast<Cut *>(w);
    p.part_ml = reinterpret_cast<float2 *>(w + kCutBytes);
    p.parts = reinterpret_cast<float *>(w + parts_offset(p.part_rows));
    // Both start early and wait inside: barriers and tensor memory are set up while the kernel before still runs.
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)blocks);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = sizeof(Smem<D>) + 1024;
    cfg.stream = s;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, attention_kernel<D>, p, kmap, vmap);
    if (e != cudaSuccess)
        return e;
    cfg.gridDim = dim3((unsigned)blocks, (unsigned)((p.part_rows + 7) / 8));
    cfg.blockDim = dim3(256);
    cfg.dynamicSmemBytes = 0;
    return cudaLaunchKernelEx(&cfg, join_kernel<D>, p);
}

dep_status_t attn_entry(const dep_attention_args_t *a, void *stream, int32_t hold = 0)
{
    if (!a || a->tokens < 0 || a->n_seq < 0 || a->Hq < 1 || a->Hk < 1 || a->Hq % a->Hk != 0 || a->page_size < 1 ||
        a->table_width < 0 || a->n_pages < 0 || a->workspace_bytes < 0 || !(a->scale >= 0.0f) || !isfinite(a->scale * kLog2e))
        return DEP_ERR_INVALID_ARG;
    if (a->D != 64 && a->D != 128)
        return DEP_ERR_UNSUPPORTED;
    if (a->n_seq == 0)
        return a->tokens == 0 ? DEP_OK : DEP_ERR_INVALID_ARG;
    if (!a->cu_seqlens && a->tokens % a->n_seq != 0)
        return DEP_ERR_INVALID_ARG;
    if (a->tokens == 0)
        return DEP_OK;
    // Lengths, rows of a sequence and channels of a token in 32 bits.
    if (a->tokens > INT32_MAX || a->tokens * a->Hq > INT32_MAX - 4096 || (int64_t)a->Hq * a->D > INT32_MAX ||
        (int64_t)a->table_width * a->page_size > INT32_MAX - 4096 || a->n_pages > INT32_MAX || a->n_seq > INT32_MAX - 4096)
        return DEP_ERR_UNSUPPORTED;
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
    p.ts = a->table_stride, p.tokens = T, p.each = T / a->n_seq, p.n_pages = cache ? a->n_pages : 0;
    p.n_seq = a->n_seq, p.Hq = a->Hq, p.Hk = a->Hk, p.G = a->Hq / a->Hk, p.page = a->page_size, p.most = a->table_width * a->page_size;
    // Division of a number below 2^31: 2^k / page rounded up, with 2^(k - 31) no less than the page.
    int k = 31;
    while ((1ll << (k - 31)) < a->page_size)
        ++k;
    p.page_shift = k, p.page_mul = (uint32_t)(((1ull << k) + a->page_size - 1) / a->page_size);
    p.scale = a->scale, p.status = a->status, p.hold = hold, p.part_rows = part_rows(T, a->Hq, a->Hk);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    // A tile in boxes that lie within a page: their slots divide both, and are whole groups of the swizzle.  (No maps of strides
    // of zero, which nothing says that a map may have.)
    int32_t box = kTile;
    while (a->page_size % box != 0)
        box /= 2;
    CUtensorMap kmap{}, vmap{};
    if (box >= 8 && cache && !kc.flat() && !vc.flat() &&
        encode_bf16_cache(&kmap, a->k_cache, a->D, a->page_size, a->Hk, a->n_pages, a->k_slot_stride, a->k_head_stride, a->k_page_stride, box) == CUDA_SUCCESS &&
        encode_bf16_cache(&vmap, a->v_cache, a->D, a->page_size, a->Hk, a->n_pages, a->v_slot_stride, a->v_head_stride, a->v_page_stride, box) == CUDA_SUCCESS)
        p.box = box;
    p.wide = o.aligned(32);
    uint8_t *const ws = static_cast<uint8_t *>(a->workspace);
    const cudaError_t e = a->D == 128 ? attn_launch<128>(p, ws, kmap, vmap, s) : attn_launch<64>(p, ws, kmap, vmap, s);
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

dep_status_t dep_attention_selftest_timeout(const dep_attention_args_t *args, int32_t code, void *stream)
{
    if (code < DEP_DEV_TIMEOUT_PRODUCER || code > DEP_DEV_TIMEOUT_EPILOGUE)
        return DEP_ERR_INVALID_ARG;
    return dep::attn_entry(args, stream, code);
}

}  // extern "C"
