// int8_gemm.cu -- the projection with 8-bit integers on both sides.
//
//     y[b, n] = bf16(x_scale[b] * w_scale[n] * sum_k x[b, k] W[n, k])
//
// This GPU's tensor cores have no fast 8-bit integer mode, but an int8 is exact in
// FP16, a product of two is an integer of at most 2^14, and 1024 of them add up to
// at most 2^24: an FP32 accumulator holds every such sum exactly, in any order.  So
// the products run as FP16 MMAs, and after at most 1024 columns the accumulators
// are drained into 32-bit integers.
//
// int8_rows_kernel<BT>, up to 4 rows, and for small products: four-way integer dot products
// on whole weight rows.  A block takes four weight rows at a time against BT batch rows; a
// thread loads 16 bytes of each weight row, one step ahead, and 16 of each batch row (which
// stay in L1), so a weight byte costs BT / 4 multiply-adds and next to nothing else.  The
// sums of a block's threads meet by warp reductions and through shared memory.
// Bound: the weight's bytes up to 2 rows, then the integer dot products (58 a cycle and SM).
// Measured: 7168 x 12288 at 1 row 14.9 us (87 % of the copy rate), 49376 x 7168 55 us (95 %), at 4
// rows 62 to 66 (80 to 84 %).
//
// int8_kernel<NT>: persistent blocks over units of 128 weight rows x 256 columns.
//   warp 0      TMA: weight stages, 32 KB of int8 each (256 consecutive bytes a row), at most two
//               copies in flight: 10 MB over all blocks cover the memory's latency, and more only
//               queue up behind each other, the copy that the block waits for among them.  (14560 x
//               7168 at 16 rows: all of 6 stages in flight 25.9 us, 3 of 4 24.2, 2 of 4 23.9, 2 of 2
//               25.1; 7168 x 12288 at 64 rows 32.7, 31.0, 30.2, 30.5.)
//   warps 2, 3  x, in slots of NT x SK columns as FP16.  Up to 32 rows they widen it
//               from the caller's int8 themselves.  Above, int8_widen_kernel has
//               written it as FP16 into the workspace (padded with zeros; the two are
//               chained by programmatic dependent launch), and warp 2 copies it by
//               TMA.  (x of 128 rows is twice the weight's bytes out of L2; sharing it
//               by multicast in clusters of two blocks cost 1 to 9 us more than it saved.)
//   CONV warps  turn a weight stage into FP16 and store it into a ring of slots of
//               tensor memory: lane = weight row, so that the operand crosses shared
//               memory once, as bytes.  A byte b becomes FP16 1024 + (b ^ 0x80) by one
//               byte permutation, and minus 1152 exactly b.
//   warp 1      issues tcgen05.mma: A = the weight, from tensor memory, B = x, from
//               shared memory, M = 128, N = NT.  Up to 64 rows a second warp (3, or the
//               last one) issues too: they take turns at the slots, each with its own accumulator.
//   EPI warps   drain the accumulators into integers, and finish tiles
// A weight slot and its x slot share one pair of barriers: an issuing thread spends
// about 64 cycles on an MMA, 55 on a commit and 100 on a wait, so one wait (tested
// ahead, while the MMAs before it are issued) and one commit a slot.
// Where whole tiles would leave blocks idle, the blocks take equal ranges of units, and
// every block stores its part of a tile that several share (integers: exact in any order);
// the one that comes last adds the parts, rounds and stores.  (Adding them by integer
// atomics took 18 us at 128 rows: about 200 billion a second.)  No block waits for another.
// Bound: up to 128 rows the latencies between the roles (1600 cycles a unit where its bytes take
// 1400), above the MMAs one after another.  Measured: 49376 x 7168 at 16 rows 63.9 us (82 % of the
// copy rate), at 128 rows 78.6; 14560 x 7168 at 16 rows 24.5, at 128 rows 33.7, at 256 rows 50 to 51
// (1060 TFLOP/s, 54 % of the BF16 rate; its draining threads spill 332 bytes).  The BF16 projection of this library,
// as eager launches in a graph like these: 49376 x 7168 at 16 rows 109 us, at 128 rows 114; 14560 x 7168 at 16 rows
// 36, at 128 rows 37, at 256 rows 44.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <new>

#include "internal.h"
#include "layer.h"
#include "ptx.cuh"

struct dep_int8_plan_s {
    int64_t N = 0, K = 0;
    int32_t max_rows = 0;
    int device = -1;
    int sm_count = 0;
    void *block = nullptr;  // device memory: status, counters, parts, x in FP16
    size_t bytes = 0;
    int *status = nullptr;
    int *counters = nullptr;  // arrivals at shared tiles, zero between launches
    int *parts = nullptr;     // parts of shared tiles
    size_t clear_bytes = 0;   // status and counters, from `block` on
    uint16_t *xh = nullptr, *bounds = nullptr;
    uint64_t wait_limit_ns = 1000000000ull;  // 1 s per wait
};

namespace dep {
namespace {

constexpr int64_t kMaxK = 131056;  // 131056 * 128 * 128 < 2^31
constexpr int kBM = 128;           // weight rows of a tile (MMA M)
constexpr int kKU = 256;           // columns of a unit
constexpr int kMaxUnits = 512;     // kMaxK / kKU, rounded up
constexpr int kWBytes = kBM * kKU; // a weight stage: two boxes of 128 columns

template <int NT>
struct Int8Shape {
    static constexpr bool DIRECT = NT <= 32;             // x comes straight from the caller
    static constexpr int CONV = NT <= 64 ? 8 : 4;        // converting warps (from warp 4 on)
    static constexpr int GROUPS = CONV / 4;              // four warps take 128 columns
    static constexpr int ISSUERS = GROUPS;               // issuer i takes the slots of group i
    static constexpr int EPI = NT > 128 ? 16 : NT > 64 ? 8 : 4;  // draining warps
    static constexpr int ISSUER1 = ISSUERS == 1 ? -1 : DIRECT ? 4 + CONV + EPI : 3;  // the second issuing warp
    static constexpr int THREADS = (4 + CONV + EPI + (ISSUER1 > 3)) * 32;
    static constexpr int COLS = NT / (EPI / 4);          // batch columns of a draining thread
    static constexpr int BUFS = NT <= 128 ? 2 : 1;       // sets of accumulators, one for each issuer
    static constexpr int SK = NT > 64 && NT <= 128 ? 128 : 64;  // columns of a slot
    static constexpr int SLOTS = NT > 128 ? 5 : NT > 64 ? 4 : 8;  // slots of tensor memory, and of x
    static constexpr int SLOT_COLS = SK / 2;             // a slot's 32-bit columns of tensor memory
    static constexpr int PER = kKU / SK;                 // slots of a unit
    static constexpr int EXACT = 1024 * ISSUERS / kKU;   // units whose sums an FP32 accumulator holds exactly
    static constexpr int X_BYTES = NT * SK * 2;          // an x slot
    static constexpr int FIT = (kMaxDynamicSmem - 1024 - 512 - (DIRECT ? 0 : 1024) - SLOTS * X_BYTES) / kWBytes;
    static constexpr int WS = FIT < 4 ? FIT : 4;         // weight stages
    static constexpr int FLIGHT = 2;                     // weight copies in flight
    static constexpr int ACC0 = 256;                     // the accumulators' first column
    static constexpr int BARS = 2 * WS + 2 * SLOTS + 2 * BUFS + 2;
    static constexpr int BOUNDS = DIRECT ? 0 : kMaxUnits * 2;  // bytes: bounds of x's units
    static constexpr int SMEM = 1024 + WS * kWBytes + SLOTS * X_BYTES + BARS * 8 + 16 + BOUNDS;
    static_assert(SLOTS * SLOT_COLS <= ACC0 && ACC0 + BUFS * ISSUERS * NT <= 512 && SMEM <= kMaxDynamicSmem, "");
    static_assert(GROUPS == 1 || (PER == 4 && SLOTS == 8), "group g: slots 2g, 2g + 1 of the four of a unit");
    // The slot after s among those of one group (and of one issuer), and whether the ring wraps.
    __device__ static bool next(int &s)
    {
        s += GROUPS == 1 || (s & 1) == 0 ? 1 : 3;
        if (s < SLOTS)
            return false;
        s -= SLOTS;
        return true;
    }
};

// How a launch deals its units out to its blocks: `whole` tiles, or single units; the
// first `rem` blocks get one more than `base` of them.
struct Int8Split {
    int tiles, units;  // units of a tile
    int blocks, whole, base, rem;
    __host__ __device__ int begin(int c) const  // block c's first unit
    {
        return (c * base + (c < rem ? c : rem)) * (whole ? units : 1);
    }
    __device__ int owner(int u) const  // the block of unit u
    {
        const uint32_t v = whole ? (uint32_t)u / (uint32_t)units : (uint32_t)u, big = (uint32_t)rem * (base + 1);
        return (int)(v < big ? v / (uint32_t)(base + 1) : rem + (v - big) / (uint32_t)base);
    }
};

// Walks a block's units [begin, end): the part of the last tile first, then from the
// first tile on, so that the parts that blocks share are done early.
struct Int8Walk {
    int begin, end, units, first, last, m;
    __device__ Int8Walk(int b, int e, int ku)
        : begin(b), end(e), units(ku), first((uint32_t)b / (uint32_t)ku), last((uint32_t)(e - 1) / (uint32_t)ku),
          m(last - first + 1)
    {
    }
    __device__ int tile(int i) const { return i == 0 ? last : first + i - 1; }
    __device__ int from(int t) const { return begin > t * units ? begin - t * units : 0; }  // units inside the tile
    __device__ int to(int t) const { return end < (t + 1) * units ? end - t * units : units; }
};

struct Int8Cursor {
    const Int8Walk &w;
    int i = 0, t, u, stop;
    __device__ explicit Int8Cursor(const Int8Walk &walk) : w(walk) { seek(); }
    __device__ void seek()
    {
        t = w.tile(i);
        u = w.from(t);
        stop = w.to(t);
    }
    __device__ bool done() const { return i >= w.m; }
    __device__ void next()
    {
        if (++u == stop && ++i < w.m)
            seek();
    }
};

struct Int8Params {
    const uint8_t *x;       // int8 [B, K]
    const uint16_t *bounds; // of x's units, where x was widened ahead
    const float *xs, *ws;
    uint16_t *y;
    int B, K;
    int64_t N;
    Int8Split split;
    int *counters, *parts;
    int *status;
    uint64_t limit_ns;
};

// True if the barrier's phase of this parity has completed; never waits.
__device__ __forceinline__ bool mbar_test(uint32_t bar, uint32_t parity)
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

// D[tmem] (+)= A[tmem] * B[smem desc]^T, FP16 inputs, FP32 accumulation.
__device__ __forceinline__ void mma_f16_ta(uint32_t d, uint32_t a, uint64_t bdesc, uint32_t idesc, uint32_t accumulate)
{
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
        "r"(a), "l"(bdesc), "r"(idesc), "r"(accumulate)
        : "memory");
}

// 32 lanes x 32 columns of tensor memory from 32 registers.
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

// Four int8 -> four FP16, exactly.
__device__ __forceinline__ void widen4(uint32_t w, uint32_t &lo, uint32_t &hi)
{
    const uint32_t u = w ^ 0x80808080u;
    const __half2 off = __half2half2(__ushort_as_half(0x6480));  // 1152
    uint32_t a = __byte_perm(u, 0x64646464u, 0x4140), b = __byte_perm(u, 0x64646464u, 0x4342);
    __half2 ha = __hsub2(*reinterpret_cast<__half2 *>(&a), off), hb = __hsub2(*reinterpret_cast<__half2 *>(&b), off);
    lo = *reinterpret_cast<uint32_t *>(&ha);
    hi = *reinterpret_cast<uint32_t *>(&hb);
}

// Add N accumulators (whole numbers of at most 2^24) from tensor memory to integers.  FAST, where
// the MMAs wait for it: the conversion instruction runs at an eighth of the rate of an addition,
// so numbers below 2^22 are read off the mantissa of their sum with 1.5 * 2^23; if any of a
// warp's is larger, that shows in the sum's exponent and the warp converts.
template <int N, bool FAST>
__device__ __forceinline__ void drain(uint32_t taddr, int *acc)
{
    static_assert(N == 8 || N == 16, "");
    uint32_t v[16];
    if (N == 16)
        tc::ld16(taddr, *reinterpret_cast<uint32_t(*)[16]>(v));
    else
        asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                     : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7])
                     : "r"(taddr));
    tc::wait_ld();
    constexpr int kMagic = 0x4B400000;  // 1.5 * 2^23
    if (FAST) {
        int seen = 0;
#pragma unroll
        for (int i = 0; i < N; ++i)
            seen |= __float_as_int(__uint_as_float(v[i]) + __int_as_float(kMagic)) ^ kMagic;
        // |value| < 2^22 <=> the sum lies in [2^23, 2^24): sign and exponent as kMagic's
        if (__all_sync(~0u, (seen & 0xFF800000) == 0)) {
#pragma unroll
            for (int i = 0; i < N; ++i)
                acc[i] += __float_as_int(__uint_as_float(v[i]) + __int_as_float(kMagic)) - kMagic;
            return;
        }
    }
#pragma unroll
    for (int i = 0; i < N; ++i)
        acc[i] += __float2int_rn(__uint_as_float(v[i]));
}

__device__ __forceinline__ void tmem_st16(uint32_t taddr, const int *v)
{
    asm volatile("tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, "
                 "%14, %15, %16};" ::"r"(taddr),
                 "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]),
                 "r"(v[9]), "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
                 : "memory");
}

// Sixteen int8 -> sixteen FP16.
__device__ __forceinline__ void widen16(uint4 v, uint4 &lo, uint4 &hi)
{
    widen4(v.x, lo.x, lo.y);
    widen4(v.y, lo.z, lo.w);
    widen4(v.z, hi.x, hi.y);
    widen4(v.w, hi.z, hi.w);
}

// x [B, K] int8 -> xh [16 gridDim.y, Kp] FP16, zeros past B and K (Kp a multiple of 256, K of 16); and for
// each unit of 256 columns and 16 rows (a block) the largest sum of |x| that a row has there.
__global__ void __launch_bounds__(256) int8_widen_kernel(const uint8_t *__restrict__ x, uint16_t *__restrict__ xh,
                                                         uint16_t *__restrict__ bounds, int B, int K, int Kp)
{
    griddep_launch_dependents();
    __shared__ int top[8];
    const int c = blockIdx.x * kKU + (threadIdx.x & 15) * 16, row = blockIdx.y * 16 + (threadIdx.x >> 4);
    uint4 v = make_uint4(0, 0, 0, 0);
    if (row < B && c < K)
        v = *reinterpret_cast<const uint4 *>(x + (int64_t)row * K + c);
    uint4 o[2];
    widen16(v, o[0], o[1]);
    uint4 *d = reinterpret_cast<uint4 *>(xh + (int64_t)row * Kp + c);
    d[0] = o[0];
    d[1] = o[1];
    unsigned s = __dp4a(__vabs4(v.x), 0x01010101u, 0u);  // |-128| is 128, unsigned
    s = __dp4a(__vabs4(v.y), 0x01010101u, s);
    s = __dp4a(__vabs4(v.z), 0x01010101u, s);
    s = __dp4a(__vabs4(v.w), 0x01010101u, s);
#pragma unroll
    for (int m = 8; m; m >>= 1)
        s += __shfl_xor_sync(~0u, s, m);
    s = max(s, __shfl_xor_sync(~0u, s, 16));
    if ((threadIdx.x & 31) == 0)
        top[threadIdx.x >> 5] = (int)s;
    __syncthreads();
    if (threadIdx.x == 0) {
        int most = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i)
            most = max(most, top[i]);
        bounds[blockIdx.y * gridDim.x + blockIdx.x] = (uint16_t)most;  // at most 256 * 128
    }
}

constexpr int kRows = 4;           // weight rows of a block's tile
constexpr int kRowThreads = 256;   // at most
constexpr int row_blocks(int bt) { return bt <= 4 ? 4 : 3; }  // blocks of an SM: what the registers allow

template <int BT>
__global__ void __launch_bounds__(kRowThreads, row_blocks(BT))
    int8_rows_kernel(const uint8_t *__restrict__ x, const float *__restrict__ xs, const uint8_t *__restrict__ W,
                     const float *__restrict__ ws, uint16_t *__restrict__ y, int B, int64_t N, int K)
{
    __shared__ int part[2][kRowThreads / 32][kRows * BT];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5, pieces = K / 16;
    const int steps = (pieces + blockDim.x - 1) / blockDim.x;
    const int64_t tiles = (N + kRows - 1) / kRows;
    const int b0 = blockIdx.y * BT;  // this block's batch rows
    B = B - b0 < BT ? B - b0 : BT;
    x += (int64_t)b0 * K;
    xs += b0;
    y += b0 * N;
    auto load = [&](int64_t tile, int c, uint4 (&v)[kRows]) {
        const uint4 *w = reinterpret_cast<const uint4 *>(W + tile * kRows * K);
#pragma unroll
        for (int r = 0; r < kRows; ++r)
            v[r] = c < pieces && tile * kRows + r < N ? __ldcs(w + r * pieces + c) : make_uint4(0, 0, 0, 0);
    };
    uint4 next[kRows];
    load(blockIdx.x, threadIdx.x, next);
    int buf = 0;
    for (int64_t tile = blockIdx.x; tile < tiles; tile += gridDim.x, buf ^= 1) {
        int acc[kRows][BT] = {};
        for (int s = 0; s < steps; ++s) {
            uint4 v[kRows];
#pragma unroll
            for (int r = 0; r < kRows; ++r)
                v[r] = next[r];
            const int c = threadIdx.x + s * blockDim.x;
            if (s + 1 < steps)
                load(tile, c + blockDim.x, next);
            else
                load(tile + gridDim.x, threadIdx.x, next);  // (past the last tile: nothing)
            if (c >= pieces)
                continue;
#pragma unroll
            for (int b = 0; b < BT; ++b) {
                if (b < B) {
                    const int4 a = __ldg(reinterpret_cast<const int4 *>(x) + b * pieces + c);
#pragma unroll
                    for (int r = 0; r < kRows; ++r) {
                        acc[r][b] = __dp4a(a.x, (int)v[r].x, acc[r][b]);
                        acc[r][b] = __dp4a(a.y, (int)v[r].y, acc[r][b]);
                        acc[r][b] = __dp4a(a.z, (int)v[r].z, acc[r][b]);
                        acc[r][b] = __dp4a(a.w, (int)v[r].w, acc[r][b]);
                    }
                }
            }
        }
#pragma unroll
        for (int r = 0; r < kRows; ++r)
#pragma unroll
            for (int b = 0; b < BT; ++b) {
                const int s = __reduce_add_sync(~0u, acc[r][b]);
                if (lane == 0)
                    part[buf][warp][r * BT + b] = s;
            }
        __syncthreads();  // (the other half of `part` is free: its readers have passed here since)
        if (threadIdx.x < kRows * BT) {
            const int r = threadIdx.x / BT, b = threadIdx.x % BT;
            const int64_t row = tile * kRows + r;
            int s = 0;
            for (int i = 0; i < warps; ++i)
                s += part[buf][i][threadIdx.x];
            if (b < B && row < N)
                y[(int64_t)b * N + row] = __bfloat16_as_ushort(__float2bfloat16_rn((float)s * (xs[b] * ws[row])));
        }
    }
}

template <int NT>
__global__ void __launch_bounds__(Int8Shape<NT>::THREADS, 1)
    int8_kernel(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmX, const Int8Params p)
{
    using S = Int8Shape<NT>;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = smem_u32(smem_raw), base = (raw + 1023u) & ~1023u;
    uint8_t *smem = smem_raw + (base - raw);
    const uint32_t w0 = base, x0 = base + S::WS * kWBytes;
    const uint32_t wfull = x0 + S::SLOTS * S::X_BYTES, wempty = wfull + 8 * S::WS;
    const uint32_t sfull = wempty + 8 * S::WS, sempty = sfull + 8 * S::SLOTS;  // a weight slot and its x slot
    const uint32_t accf = sempty + 8 * S::SLOTS, acce = accf + 8 * S::BUFS, done = acce + 8 * S::BUFS, known = done + 8;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + (known + 8 - base));
    volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);
    uint16_t *bounds = reinterpret_cast<uint16_t *>(tmem_slot + 4);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int c = blockIdx.x, KU = p.split.units;
    const Int8Walk walk(p.split.begin(c), p.split.begin(c + 1), KU);

    // Weight copies (thread 0); the first ones start before anything else is set up.
    Int8Cursor wcur(walk);
    int wst = 0;
    auto copy_w = [&](uint64_t pol) {
        const int row = wcur.t * kBM, col = wcur.u * kKU;
        const uint32_t dst = w0 + wst * kWBytes, bar = wfull + 8 * wst;
        mbar_arrive_expect_tx(bar, kWBytes);
        tma_load_2d(dst, &tmW, col, row, bar, pol);
        tma_load_2d(dst + kWBytes / 2, &tmW, col + 128, row, bar, pol);
        wcur.next();
        ++wst;
    };
    if (threadIdx.x == 0) {
        for (int i = 0; i < S::WS; ++i)
            mbar_init(wfull + 8 * i, 1);
        fence_mbar_init();
        const uint64_t pol = policy_evict_first();
        while (wst < S::FLIGHT && !wcur.done())
            copy_w(pol);
        *abort_flag = 0;
    }
    if (warp == 2) {
        auto init = [&](uint32_t bar, int n, int count) {
            for (int i = lane; i < n; i += 32)
                mbar_init(bar + 8 * i, count);
        };
        init(wempty, S::WS, S::CONV);
        init(sfull, S::SLOTS, 4 + 1);  // four converting warps, and x
        init(sempty, S::SLOTS, 1);       // its MMAs
        init(accf, S::BUFS, S::ISSUERS);
        init(acce, S::BUFS, S::EPI);
        init(done, 1, S::ISSUERS);
        init(known, 1, 1);
        fence_mbar_init();
    }
    if (warp == 1) {
        tc::alloc(smem_u32(tmem_slot), 512);
        tc::relinquish();
    }
    tc::fence_before();
    __syncthreads();
    tc::fence_after();
    const uint32_t tmem = *tmem_slot;
    auto give_up = [&](int code) {
        record_status(p.status, code);
        *abort_flag = 1;
    };

    // The end of the run of units from u on (of `end`) that accumulators hold exactly: 1024 columns for each
    // issuer; or, where the bounds are known, as many as keep the sum of |x| 128 within 2^24.
    auto run_end = [&](int u, int end) {
        if (S::DIRECT)
            return u + S::EXACT < end ? u + S::EXACT : end;
        int sum = 0;
        while (u < end && (sum += bounds[u]) <= (1 << 24) / 128)
            ++u;
        return u;
    };

    if (warp == 0) {
        // ---------------- weight copies ----------------
        if (lane == 0) {
            const uint64_t pol = policy_evict_first();
            int flying = wst, first = 0;  // copies in flight, and the stage of the first of them
            uint32_t ph = 0, first_ph = 0;
            auto arrived = [&] {
                const bool ok = mbar_wait(wfull + 8 * first, first_ph, p.limit_ns);
                --flying;
                if (++first == S::WS) {
                    first = 0;
                    first_ph ^= 1u;
                }
                return ok;
            };
            if (wst == S::WS) {
                wst = 0;
                ph = 1;
            }
            while (!wcur.done()) {
                if (*abort_flag)
                    break;
                if ((flying == S::FLIGHT && !arrived()) || !mbar_wait(wempty + 8 * wst, ph ^ 1u, p.limit_ns)) {
                    give_up(DEP_DEV_TIMEOUT_PRODUCER);
                    break;
                }
                copy_w(pol);
                ++flying;
                if (wst == S::WS) {
                    wst = 0;
                    ph ^= 1u;
                }
            }
            while (flying > 0)
                if (!arrived())
                    record_status(p.status, DEP_DEV_TIMEOUT_PRODUCER);
        }
    } else if (S::DIRECT && (warp == 2 || warp == 3)) {
        // ---------------- x, widened here: each warp 128 columns of a unit ----------------
        constexpr int V = NT / 4;  // 16-byte pieces a lane: piece i is chunk (lane % 8) of row 4 i + lane / 8
        uint4 v[V];
        Int8Cursor cur(walk);
        auto fetch = [&]() {
            const int k = cur.u * kKU + (warp - 2) * 128 + (lane & 7) * 16;
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const int row = 4 * i + (lane >> 3);
                v[i] = row < p.B && k < p.K ? __ldg(reinterpret_cast<const uint4 *>(p.x + (int64_t)row * p.K + k))
                                            : make_uint4(0, 0, 0, 0);
            }
        };
        int s = 2 * (warp - 2);  // slots s and s + 1: 64 columns each
        uint32_t ph = 0;
        fetch();
        while (!cur.done()) {
            const bool ok = !*abort_flag && mbar_wait(sempty + 8 * s, ph ^ 1u, p.limit_ns) &&
                            mbar_wait(sempty + 8 * s + 8, ph ^ 1u, p.limit_ns);
            if (!__all_sync(~0u, ok)) {
                if (lane == 0)
                    give_up(DEP_DEV_TIMEOUT_PRODUCER);
                break;
            }
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const int row = 4 * i + (lane >> 3), ch = lane & 7;
                uint4 lo, hi;
                widen16(v[i], lo, hi);
                // rows of 128 bytes, 16-byte pieces in the 128-byte swizzle
                const uint32_t at = x0 + (s + (ch >> 2)) * S::X_BYTES + row * 128;
                const uint32_t a0 = at + (((ch & 3) * 2) ^ (row & 7)) * 16, a1 = at + (((ch & 3) * 2 + 1) ^ (row & 7)) * 16;
                asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(a0), "r"(lo.x), "r"(lo.y), "r"(lo.z), "r"(lo.w)
                             : "memory");
                asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(a1), "r"(hi.x), "r"(hi.y), "r"(hi.z), "r"(hi.w)
                             : "memory");
            }
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");  // the MMA reads through the async proxy
            __syncwarp();
            if (lane < 2)
                mbar_arrive(sfull + 8 * (s + lane));
            cur.next();
            if (!cur.done())
                fetch();
            s ^= 4;
            ph ^= (uint32_t)((s & 4) == 0);
        }
    } else if (!S::DIRECT && warp == 2) {
        // ---------------- x copies ----------------
        if (lane == 0) {
            prefetch_tmap(&tmX);
            const uint64_t pol = policy_evict_last();
            griddep_wait();  // x in FP16 is written by the preceding grid
            Int8Cursor cur(walk);
            int s = 0;
            uint32_t ph = 0;
            int64_t issued = 0;
            bool ok = true;
            for (; ok && !cur.done(); cur.next()) {
                for (int h = 0; h < S::PER; ++h) {
                    if (*abort_flag || !mbar_wait(sempty + 8 * s, ph ^ 1u, p.limit_ns)) {
                        give_up(DEP_DEV_TIMEOUT_PRODUCER);
                        ok = false;
                        break;
                    }
                    mbar_arrive_expect_tx(sfull + 8 * s, S::X_BYTES);
                    const int block64 = cur.u * (kKU / 64) + h * (S::SK / 64);
                    tma_load_3d(x0 + s * S::X_BYTES, &tmX, 0, 0, block64, sfull + 8 * s, pol);
                    ++issued;
                    if (++s == S::SLOTS) {
                        s = 0;
                        ph ^= 1u;
                    }
                }
            }
            for (int64_t i = issued < S::SLOTS ? issued : S::SLOTS; i > 0; --i) {
                if (--s < 0) {
                    s = S::SLOTS - 1;
                    ph ^= 1u;
                }
                if (!mbar_wait(sempty + 8 * s, ph, p.limit_ns))  // copied, and consumed
                    record_status(p.status, DEP_DEV_TIMEOUT_PRODUCER);
            }
        }
    } else if (warp == 1 || warp == S::ISSUER1) {
        // ---------------- MMA issue ----------------
        const int mi = warp == 1 ? 0 : 1;
        if (lane == 0) {
            // FP16 operands (format 0), FP32 accumulator, N >> 3 and M >> 4
            constexpr uint32_t idesc = (1u << 4) | ((uint32_t)(NT >> 3) << 17) | ((uint32_t)(kBM >> 4) << 24);
            int s = 2 * mi, buf = 0;
            uint32_t sph = 0, bph = 0;
            bool ok = S::DIRECT || mbar_wait(known, 0, p.limit_ns), ready = false;
            if (!ok)
                give_up(DEP_DEV_TIMEOUT_MMA);
            for (int seg = 0; seg < walk.m && ok; ++seg) {
                const int t = walk.tile(seg), end = walk.to(t);
                for (int u = walk.from(t); u < end && ok;) {
                    const int stop = run_end(u, end);
                    if (!mbar_wait(acce + 8 * buf, bph ^ 1u, p.limit_ns)) {
                        give_up(DEP_DEV_TIMEOUT_MMA);
                        ok = false;
                        break;
                    }
                    tc::fence_after();
                    const uint32_t d = tmem + (uint32_t)(S::ACC0 + (buf * S::ISSUERS + mi) * NT);
                    uint32_t accumulate = 0;
                    for (int n = (stop - u) * (S::PER / S::ISSUERS); n > 0; --n) {
                        if (!ready && (*abort_flag || !mbar_wait(sfull + 8 * s, sph, p.limit_ns))) {
                            give_up(DEP_DEV_TIMEOUT_MMA);
                            ok = false;
                            break;
                        }
                        tc::fence_after();
                        const uint32_t a = tmem + (uint32_t)(s * S::SLOT_COLS), freed = sempty + 8 * s;
                        const uint64_t b = tc::desc_sw128(x0 + (uint32_t)(s * S::X_BYTES));
                        sph ^= (uint32_t)S::next(s);
                        ready = mbar_test(sfull + 8 * s, sph);  // the next slot's
#pragma unroll
                        for (int i = 0; i < S::SK / 16; ++i) {
                            mma_f16_ta(d, a + 8 * i, b + (uint64_t)(((i / 4) * NT * 128) >> 4) + 2 * (i % 4), idesc,
                                       accumulate);
                            accumulate = 1;
                        }
                        tc::commit(freed);
                    }
                    if (!ok)
                        break;
                    u = stop;
                    tc::commit(accf + 8 * buf);
                    if (++buf == S::BUFS) {
                        buf = 0;
                        bph ^= 1u;
                    }
                }
            }
            tc::commit(done);  // tensor memory is freed at the end: wait for every MMA
            if (!mbar_wait(done, 0, p.limit_ns))
                record_status(p.status, DEP_DEV_TIMEOUT_MMA);
        }
    } else if (warp >= 4 && warp < 4 + S::CONV) {
        // ---------------- int8 -> FP16 into tensor memory ----------------
        const int wg = (warp - 4) >> 2, q = warp & 3, row = 32 * q + lane;
        const int n_units = walk.end - walk.begin;
        int ws = 0, s = 2 * wg;  // two groups: group g takes columns [128 g, 128 g + 128) of every stage
        uint32_t wph = 0, sph = 0;
        for (int i = 0; i < n_units; ++i) {
            bool ok = !*abort_flag && mbar_wait(wfull + 8 * ws, wph, p.limit_ns);
            const uint32_t src = w0 + (uint32_t)(ws * kWBytes + wg * (kWBytes / 2) + row * 128);
#pragma unroll
            for (int h = 0; h < 4 / S::GROUPS; ++h) {  // 64 columns
                if (S::SK == 64 || h % 2 == 0) {
                    ok = ok && mbar_wait(sempty + 8 * s, sph ^ 1u, p.limit_ns);
                    if (!__all_sync(~0u, ok))
                        break;
                    tc::fence_after();
                }
                uint32_t v[32];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    uint32_t w[4];
                    const uint32_t at =
                        src + (uint32_t)((h / 2) * (kWBytes / 2) + ((4 * (h % 2) + j) ^ (row & 7)) * 16);
                    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                                 : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3])
                                 : "r"(at));
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        widen4(w[e], v[8 * j + 2 * e], v[8 * j + 2 * e + 1]);
                }
                tmem_st32(tmem + ((uint32_t)(32 * q) << 16) +
                              (uint32_t)(s * S::SLOT_COLS + (S::SK == 64 ? 0 : 32 * (h % 2))),
                          v);
                if (h == 4 / S::GROUPS - 1) {
                    __syncwarp();
                    if (lane == 0)
                        mbar_arrive(wempty + 8 * ws);
                }
                if (S::SK == 64 || h % 2 == 1) {
                    tmem_wait_st();
                    tc::fence_before();
                    __syncwarp();
                    if (lane == 0)
                        mbar_arrive(sfull + 8 * s);
                    sph ^= (uint32_t)S::next(s);
                }
            }
            if (!__all_sync(~0u, ok)) {
                if (lane == 0)
                    give_up(DEP_DEV_TIMEOUT_CONSUMER);
                break;
            }
            if (++ws == S::WS) {
                ws = 0;
                wph ^= 1u;
            }
        }
    } else if (warp >= 4 + S::CONV) {
        // ---------------- drain and finish ----------------
        const int e = warp - 4 - S::CONV, q = warp & 3, c0 = (e / 4) * S::COLS;
        const uint32_t lane_addr = tmem + ((uint32_t)(32 * q) << 16) + (uint32_t)(S::ACC0 + c0);
        const int cols = p.B - c0 < S::COLS ? p.B - c0 : S::COLS;  // of these, columns of the batch (may be <= 0)
        int buf = 0;
        uint32_t bph = 0;
        if (!S::DIRECT && e == 0) {  // bounds of x's units, for the issuers and the other draining warps
            griddep_wait();
            for (int i = lane; i < KU; i += 32) {
                int most = 0;
                for (int r = 0; r * 16 < p.B; ++r)
                    most = max(most, (int)p.bounds[r * KU + i]);
                bounds[i] = (uint16_t)most;
            }
            __syncwarp();
            if (lane == 0)
                mbar_arrive(known);
        }
        bool ok = __all_sync(~0u, S::DIRECT || mbar_wait(known, 0, p.limit_ns));
        if (!ok && lane == 0)
            give_up(DEP_DEV_TIMEOUT_EPILOGUE);
        for (int seg = 0; seg < walk.m && ok; ++seg) {
            const int t = walk.tile(seg), end = walk.to(t);
            const int64_t n = (int64_t)t * kBM + 32 * q + lane;
            const float ws = n < p.N ? p.ws[n] : 0.0f;
            int acc[S::COLS];
#pragma unroll
            for (int j = 0; j < S::COLS; ++j)
                acc[j] = 0;
            for (int u = walk.from(t); u < end;) {
                ok = __all_sync(~0u, mbar_wait(accf + 8 * buf, bph, p.limit_ns));
                if (!ok) {
                    if (lane == 0)
                        give_up(DEP_DEV_TIMEOUT_EPILOGUE);
                    break;
                }
                tc::fence_after();
                constexpr int D = NT > 128 ? 8 : 16;  // columns at a time: what the registers allow
#pragma unroll
                for (int j = 0; j < S::COLS; j += D)
                    if (j < cols)
#pragma unroll
                        for (int m = 0; m < S::ISSUERS; ++m)
                            drain<D, (NT > 128)>(lane_addr + (uint32_t)((buf * S::ISSUERS + m) * NT + j), acc + j);
                u = run_end(u, end);
                if (u < end) {
                    tc::fence_before();
                    __syncwarp();
                    if (lane == 0)
                        mbar_arrive(acce + 8 * buf);
                    if (++buf == S::BUFS) {
                        buf = 0;
                        bph ^= 1u;
                    }
                }
            }
            if (!ok)
                break;
            // The tile's end runs once or twice: its code, if unrolled over the columns, would cost more to fetch
            // than to run.  So the sums go back over the accumulators, and loops read them from there.
            const uint32_t back = lane_addr + (uint32_t)(buf * S::ISSUERS * NT);
#pragma unroll
            for (int j = 0; j < S::COLS; j += 16)
                if (j < cols)
                    tmem_st16(back + j, acc + j);
            tmem_wait_st();
            // A tile that several blocks share: each stores its part, and the one that comes last adds them.
            bool last = true;
            const int ca = p.split.owner(t * KU), parts = p.split.owner((t + 1) * KU - 1) - ca + 1;
            const auto part = [&](int b) {  // this warp's part of block b's
                const int slot = p.split.begin(b) > t * KU ? 0 : 1;  // the tile that its range starts in, or the last
                return p.parts + (((int64_t)b * 2 + slot) * NT + c0) * kBM + 32 * q + lane;
            };
            if (parts > 1) {
                int *mine = part(c);
#pragma unroll 1
                for (int j = 0; j < cols; j += 16) {
                    uint32_t v[16];
                    tc::ld16(back + j, v);
                    tc::wait_ld();
#pragma unroll
                    for (int i = 0; i < 16; ++i)
                        __stcg(mine + (j + i) * kBM, (int)v[i]);
                }
                __threadfence();
                __syncwarp();
                int old = 0;
                if (lane == 0)
                    old = atomicAdd(p.counters + t * 16 + e, 1);
                last = __shfl_sync(~0u, old, 0) == parts - 1;
                if (last) {
                    __threadfence();
                    if (lane == 0)
                        p.counters[t * 16 + e] = 0;
                }
            }
            if (last) {
                uint16_t *y = p.y + (int64_t)c0 * p.N + n;
#pragma unroll 1
                for (int j = 0; j < cols; j += 16, y += 16 * p.N) {
                    uint32_t v[16];
                    tc::ld16(back + j, v);
                    tc::wait_ld();
#pragma unroll 1
                    for (int i0 = 0; i0 < parts; i0 += 2) {  // two parts in flight; this block's own is there already
                        const int a0 = ca + i0, a1 = a0 + 1;
                        const bool in0 = a0 != c, in1 = i0 + 1 < parts && a1 != c;
                        const int *s0 = part(in0 ? a0 : c) + j * kBM, *s1 = part(in1 ? a1 : c) + j * kBM;
                        if (parts == 1)
                            break;
                        int u0[16], u1[16];
#pragma unroll
                        for (int i = 0; i < 16; ++i) {
                            u0[i] = in0 ? __ldcg(s0 + i * kBM) : 0;
                            u1[i] = in1 ? __ldcg(s1 + i * kBM) : 0;
                        }
#pragma unroll
                        for (int i = 0; i < 16; ++i)
                            v[i] += u0[i] + u1[i];
                    }
                    const float xs = j + (lane & 15) < cols ? p.xs[c0 + j + (lane & 15)] : 0.0f;
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        const float scale = __shfl_sync(~0u, xs, i) * ws;
                        if (j + i < cols && n < p.N)
                            y[i * p.N] = __bfloat16_as_ushort(__float2bfloat16_rn((float)(int)v[i] * scale));
                    }
                }
            }
            tc::fence_before();
            __syncwarp();
            if (lane == 0)
                mbar_arrive(acce + 8 * buf);
            if (++buf == S::BUFS) {
                buf = 0;
                bph ^= 1u;
            }
        }
    }

    __syncwarp();
    tc::fence_before();
    __syncthreads();
    if (warp == 1) {
        tc::fence_after();
        tc::dealloc(tmem, 512);
    }
}

// MMA width of a pass of B rows.
// NT: the least that holds the batch.  (96 instead of 128: 14560 x 7168 at 96 rows 33.0 -> 31.7 us; 192 instead of
// 256: at 192 rows 48.3 -> 44.5.)
constexpr int kWidths[] = {16, 32, 64, 96, 128, 192, 256};
int width(int32_t B)
{
    int i = 0;
    while (kWidths[i] < B && kWidths[i] < 256)
        ++i;
    return kWidths[i];
}

Int8Split split_for(int64_t N, int64_t K, int nt, int sms)
{
    Int8Split s;
    s.tiles = (int)((N + kBM - 1) / kBM);
    s.units = (int)((K + kKU - 1) / kKU);
    const int all = s.tiles * s.units, waves = (s.tiles + sms - 1) / sms;
    // Equal ranges, of about four units or more, unless whole tiles keep enough of the blocks busy: nearly all, or, above
    // 128 rows, where a part of a tile is 96 or 128 KB, 70 %.  Equal ranges and whole tiles, 14560 x 7168 (75 %): 23.9
    // and 26.8 us at 16 rows, 33.6 and 34.7 at 128, 44.3 and 44.4 at 192, 52.1 and 50.9 at 256; 16384 x 4096 (84 %):
    // 35.5 and 30.6 at 192, 43.3 and 36.8 at 256; 7168 x 12288 (37 %): 61.5 and 84 at 256.
    s.whole = s.tiles * 100ll >= (int64_t)waves * sms * (nt > 128 ? 70 : 95);
    const int n = s.whole ? s.tiles : all, c = s.whole ? n : (all + 3) / 4;
    s.blocks = c < sms ? c : sms;
    s.base = n / s.blocks;
    s.rem = n % s.blocks;
    return s;
}

template <int NT>
cudaError_t int8_prepare()
{
    static std::atomic<uint64_t> devices{0};
    return set_smem_attr(int8_kernel<NT>, devices);
}

template <int NT>
cudaError_t int8_launch(const dep_int8_plan_s &pl, const void *W, const Int8Params &p, cudaStream_t stream)
{
    using S = Int8Shape<NT>;
    cudaError_t e = int8_prepare<NT>();
    if (e != cudaSuccess)
        return e;
    CUtensorMap tmW, tmX;
    if (encode_u8_2d(&tmW, W, (uint64_t)pl.K, (uint64_t)pl.N, 128, kBM) != CUDA_SUCCESS)
        return cudaErrorInvalidValue;
    if (S::DIRECT)
        tmX = tmW;  // not used
    else if (encode_bf16_3d_blocks(&tmX, pl.xh, (uint64_t)(p.split.units * kKU), NT, NT, S::SK / 64) != CUDA_SUCCESS)
        return cudaErrorInvalidValue;
    return launch(int8_kernel<NT>, dim3(p.split.blocks), dim3(S::THREADS), (size_t)S::SMEM, stream,
                  !S::DIRECT /* after int8_widen_kernel */, tmW, tmX, p);
}

template <int BT>
cudaError_t rows_launch(const dep_int8_plan_s &pl, const uint8_t *x, const float *xs, const void *W, const float *ws,
                        uint16_t *y, int32_t B, cudaStream_t stream)
{
    const int32_t groups = (B + BT - 1) / BT;
    const int64_t tiles = (pl.N + kRows - 1) / kRows, room = (int64_t)pl.sm_count * row_blocks(BT) / groups,
                  most = room < 1 ? 1 : room;
    // As many threads as share a row's pieces most evenly.
    const int pieces = (int)(pl.K / 16);
    int threads = kRowThreads;
    for (int n = kRowThreads - 32; n >= kRowThreads / 2; n -= 32)
        if ((pieces + n - 1) / n * n < (pieces + threads - 1) / threads * threads)
            threads = n;
    int8_rows_kernel<BT><<<dim3((unsigned)(tiles < most ? tiles : most), (unsigned)groups), threads, 0, stream>>>(
        x, xs, static_cast<const uint8_t *>(W), ws, y, B, pl.N, (int)pl.K);
    return cudaGetLastError();
}

cudaError_t int8_pass(const dep_int8_plan_s &pl, const uint8_t *x, const float *xs, const void *W, const float *ws,
                      uint16_t *y, int32_t B, cudaStream_t stream)
{
    // Dot products, or tensor cores: 14560 x 7168, 21 and 26 us at 4 rows, 27.5 and 26 at 5; 49376 x 7168, 62 and 66 us
    // at 4 rows, 83 and 66 at 5.  Small products have the shorter way through dot products, and read the weight once for
    // every 8 rows: 7168 x 12288, 22 and 24 us at 5 rows; 2311 x 3056, 9 and 10 us at 16, 11.5 and 10.5 at 24.
    if (B <= 4 || (double)pl.N * (double)pl.K * B * ((B + 7) / 8) < 5e8)
        return B == 1   ? rows_launch<1>(pl, x, xs, W, ws, y, B, stream)
               : B == 2 ? rows_launch<2>(pl, x, xs, W, ws, y, B, stream)
               : B <= 4 ? rows_launch<4>(pl, x, xs, W, ws, y, B, stream)
                        : rows_launch<8>(pl, x, xs, W, ws, y, B, stream);
    const int nt = width(B);
    const Int8Split split = split_for(pl.N, pl.K, nt, pl.sm_count);
    if (nt > 32) {
        const int Kp = (int)split.units * kKU;
        int8_widen_kernel<<<dim3((unsigned)split.units, (unsigned)(nt / 16)), 256, 0, stream>>>(x, pl.xh, pl.bounds, B,
                                                                                                (int)pl.K, Kp);
        const cudaError_t e = cudaGetLastError();
        if (e != cudaSuccess)
            return e;
    }
    const Int8Params p{x, pl.bounds, xs, ws, y, B, (int)pl.K, pl.N, split, pl.counters, pl.parts, pl.status, pl.wait_limit_ns};
    switch (nt) {
    case 16: return int8_launch<16>(pl, W, p, stream);
    case 32: return int8_launch<32>(pl, W, p, stream);
    case 64: return int8_launch<64>(pl, W, p, stream);
    case 96: return int8_launch<96>(pl, W, p, stream);
    case 128: return int8_launch<128>(pl, W, p, stream);
    case 192: return int8_launch<192>(pl, W, p, stream);
    default: return int8_launch<256>(pl, W, p, stream);
    }
}

// Raise every kernel's shared-memory limit now, so that no first launch does it inside a capture.
cudaError_t int8_prepare_device()
{
    // The same split of L1 and shared memory as the kernel it is chained to: no SM has to drain between them.
    cudaError_t c = cudaFuncSetAttribute(int8_widen_kernel, cudaFuncAttributePreferredSharedMemoryCarveout,
                                         (int)cudaSharedmemCarveoutMaxShared);
    if (c != cudaSuccess)
        return c;
    for (cudaError_t e : {int8_prepare<16>(), int8_prepare<32>(), int8_prepare<64>(), int8_prepare<96>(),
                          int8_prepare<128>(), int8_prepare<192>(), int8_prepare<256>()})
        if (e != cudaSuccess)
            return e;
    return cudaSuccess;
}

}  // namespace
}  // namespace dep

extern "C" {

dep_status_t dep_int8_plan(int64_t N, int64_t K, int32_t max_rows, dep_int8_plan_t *out)
{
    if (!out)
        return DEP_ERR_INVALID_ARG;
    *out = nullptr;
    if (N < 1 || K < 16 || max_rows < 1)
        return DEP_ERR_INVALID_ARG;
    if (K % 16 != 0)
        return DEP_ERR_MISALIGNED;
    if (K > dep::kMaxK || N > INT32_MAX || (N / dep::kBM + 2) * (K / dep::kKU + 1) > INT32_MAX)
        return DEP_ERR_UNSUPPORTED;
    dep_int8_plan_s *p = new (std::nothrow) dep_int8_plan_s;
    if (!p)
        return DEP_ERR_OOM;
    p->N = N;
    p->K = K;
    p->max_rows = max_rows;
    cudaDeviceProp prop;
    if (cudaGetDevice(&p->device) != cudaSuccess || cudaGetDeviceProperties(&prop, p->device) != cudaSuccess) {
        cudaGetLastError();
        delete p;
        return DEP_ERR_CUDA;
    }
    p->sm_count = prop.multiProcessorCount;
    if (prop.major * 10 + prop.minor < 100) {
        delete p;
        return DEP_ERR_UNSUPPORTED;
    }
    if (dep::int8_prepare_device() != cudaSuccess) {
        cudaGetLastError();
        delete p;
        return DEP_ERR_CUDA;
    }
    // One block of device memory: status word, counters, parts of shared tiles, x in FP16.
    const int64_t tiles = (N + dep::kBM - 1) / dep::kBM, Kp = (K + dep::kKU - 1) / dep::kKU * dep::kKU;
    const int nt = dep::width(max_rows);
    size_t parts = 0;
    for (const int w : dep::kWidths) {
        if (w > nt)
            break;
        const dep::Int8Split s = dep::split_for(N, K, w, p->sm_count);
        if (!s.whole)  // two for each block
            parts = (size_t)s.blocks * 2 * w * dep::kBM * sizeof(int);
    }
    const size_t counters = ((size_t)tiles * 16 * sizeof(int) + 255) / 256 * 256;
    p->clear_bytes = 256 + counters;
    p->bytes = p->clear_bytes + parts + (nt > 32 ? (size_t)(nt + 1) * Kp * 2 : 0);
    if (cudaMalloc(&p->block, p->bytes) != cudaSuccess) {
        cudaGetLastError();
        delete p;
        return DEP_ERR_OOM;
    }
    if (cudaMemset(p->block, 0, p->bytes) != cudaSuccess || cudaDeviceSynchronize() != cudaSuccess) {
        cudaGetLastError();
        cudaFree(p->block);
        delete p;
        return DEP_ERR_CUDA;
    }
    uint8_t *at = static_cast<uint8_t *>(p->block);
    p->status = reinterpret_cast<int *>(at);
    p->counters = reinterpret_cast<int *>(at + 256);
    p->parts = reinterpret_cast<int *>(at + p->clear_bytes);
    p->xh = reinterpret_cast<uint16_t *>(at + p->clear_bytes + parts);
    p->bounds = p->xh + (size_t)nt * Kp;  // one for each unit and 16 rows
    *out = p;
    return DEP_OK;
}

dep_status_t dep_int8_run(dep_int8_plan_t p, const void *x, const float *x_scale, const void *W, const float *w_scale,
                          void *y, int32_t B, void *stream)
{
    if (!p || B < 0)
        return DEP_ERR_INVALID_ARG;
    if (B == 0)
        return DEP_OK;
    if (!x || !x_scale || !W || !w_scale || !y)
        return DEP_ERR_INVALID_ARG;
    if (!dep::aligned(x, 16) || !dep::aligned(W, 16) || !dep::aligned(y, 16) || !dep::aligned(x_scale, 4) ||
        !dep::aligned(w_scale, 4))
        return DEP_ERR_MISALIGNED;
    const dep::Rows ry{y, 2 * (int64_t)B * p->N, 0, 1}, rx{x, B * p->K, 0, 1}, rw{W, p->N * p->K, 0, 1},
        rxs{x_scale, 4 * (int64_t)B, 0, 1}, rws{w_scale, 4 * p->N, 0, 1};
    if (overlap(ry, rx) || overlap(ry, rw) || overlap(ry, rxs) || overlap(ry, rws))
        return DEP_ERR_INVALID_ARG;
    int dev = -1;
    if (cudaGetDevice(&dev) != cudaSuccess || dev != p->device) {
        cudaGetLastError();
        return DEP_ERR_INVALID_ARG;
    }
    const int32_t step = dep::width(p->max_rows);  // rows of a pass
    for (int64_t r0 = 0; r0 < B; r0 += step) {  // (up to step - 1 beyond B, and B may be the largest int32)
        const int32_t rows = B - r0 < step ? (int32_t)(B - r0) : step;
        if (dep::int8_pass(*p, static_cast<const uint8_t *>(x) + r0 * p->K, x_scale + r0, W, w_scale,
                           static_cast<uint16_t *>(y) + r0 * p->N, rows,
                           static_cast<cudaStream_t>(stream)) != cudaSuccess) {
            cudaGetLastError();
            return DEP_ERR_CUDA;
        }
    }
    return DEP_OK;
}

dep_status_t dep_int8_plan_workspace(dep_int8_plan_t p, size_t *bytes)
{
    if (!p || !bytes)
        return DEP_ERR_INVALID_ARG;
    *bytes = p->bytes;
    return DEP_OK;
}

dep_status_t dep_int8_device_status(dep_int8_plan_t p, void *stream, int32_t *code)
{
    if (!p || !code)
        return DEP_ERR_INVALID_ARG;
    *code = 0;
    int h = 0;
    if (cudaStreamSynchronize(static_cast<cudaStream_t>(stream)) != cudaSuccess ||
        cudaMemcpy(&h, p->status, sizeof(int), cudaMemcpyDeviceToHost) != cudaSuccess) {
        cudaGetLastError();
        return DEP_ERR_CUDA;
    }
    // After a give-up counters may be left mid-protocol: clear them.
    if (h && (cudaDeviceSynchronize() != cudaSuccess || cudaMemset(p->block, 0, p->clear_bytes) != cudaSuccess)) {
        cudaGetLastError();
        return DEP_ERR_CUDA;
    }
    *code = h;
    return h ? DEP_ERR_TIMEOUT : DEP_OK;
}

void dep_int8_plan_destroy(dep_int8_plan_t p)
{
    if (!p)
        return;
    int dev = -1;
    cudaGetDevice(&dev);
    if (dev != p->device)
        cudaSetDevice(p->device);
    cudaFree(p->block);  // waits for the device's work
    if (dev >= 0 && dev != p->device)
        cudaSetDevice(dev);
    cudaGetLastError();
    delete p;
}

}  // extern "C"
