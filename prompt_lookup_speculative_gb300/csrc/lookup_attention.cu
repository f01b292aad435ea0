// lookup_attention.cu -- attention of a verify block over the paged cache.
//
// The contract is in include/lookup_target.h (lookup_paged_attention).
//
// The mathematics: out = sum_j p_j v_j / sum_j p_j with p_j = 2^(c q.k_j - c m),
// c = |scale| log2(e) (a negative scale is folded into q, exactly), in one pass over
// the cache with a running m per row: the sums so far are brought to a larger m by
// one factor.  m follows the row's maximum only when that is more than 2^8 ahead:
// p then stays within 2^8, which neither type's range nor its relative rounding
// notices, and most tiles need no correction of the sums.
//
// What bounds it: the cache's bytes, read once.  The block's N tokens and the G =
// Hq / Hkv query heads of one key-value head share every key they read, so their
// N * G rows form the M = 128 rows of tcgen05 products (16 tokens of 8 heads fill
// them exactly; fewer rows leave lanes idle, which costs no bytes): S = Q K^T of 128
// rows by a tile of 64 or 128 positions into tensor memory, softmax by one thread per
// row, P back into tensor memory, O += P V from there.  P is rounded to the cache's type,
// as the product's operand has to be (relative 2^-8 in bfloat16, 2^-11 in float16, as an
// output is); the sum takes the weights before that, and S, O, m and the sum are float32.
// float16's weights are taken 2^7 higher, for which there is room above 2^8: those down to
// 2^-21 of m's keep that rounding, and only below 2^-32 do they leave the product (2^-14
// and 2^-25 without: behind one score 17 above it, a long even tail counted 1.4 times).
//
// Few rows: the tile has idle rows, and only the warps of the live ones have a softmax
// to do, one SM quarter per 32 rows.  So a block of at most 64 (32) rows is in the tile
// two (four) times, and each copy's threads take a half (a quarter) of the columns:
// every quarter of the SM works, and a tile's softmax takes a half (a quarter) of the
// time.  The product of 16 positions goes into their copy's lanes only, and the
// copies' sums are added at the item's end.
//
// Split: the work of all requests, heads and row tiles is laid end to end in units
// of a tile and cut into equal contiguous ranges, one per CTA (two CTAs per
// SM), so that neither ragged lengths nor few requests leave an SM without work.
// A CTA finds its range from kv_len and q_len on the device.  An item that lies in
// one range is finished there; the parts of one that is cut go to the workspace and
// join_kernel adds them, in the order of the ranges: no atomics, the same bits every
// time.
//
// Short items: what runs once per item, at its begin and end, waits for its instructions
// more than for anything else, so that code is kept small: loops there are rolled, one
// copy of each step.  The next item's Q and first page ids are loaded during an item.
// 2048 items of 1 to 2048 positions, 4 heads each at D = 128: 138 us before, 83 with that
// (3.9 TB/s, 57% of a copy's rate).
//
// Long ones: 64 blocks of 16 tokens over 25000 positions, 32 heads on 4 at D = 128, 505 us
// (6.5 TB/s, 96% of a copy's rate), one token each over 12000 to 25000 667 us (7.0 TB/s).
// 16 blocks of 8 over 512 to 262144, 14 heads on 2 at D = 64, 79 us (5.0 TB/s): the
// instructions that issue a tile's products take as long as its 32 KB.  One token over 4096
// positions 15.3 us: the way through both kernels, once.  64 requests of 12000 to 25000 at
// D = 256, 16 heads on 4: 673 us with one token, 697 with blocks of 16 (6.8 TB/s).
//
// Blocks of more than 128 rows (prompts): each row tile walks the whole request's tiles, not
// its own rows' only.  8191 tokens, 32 heads on 8: 1.72 ms, with or without a window of 500.

#include "lookup_draft.h"
#include "lookup_target.h"
#include "common.cuh"

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstdint>
#include <type_traits>

namespace {

using lkd::allow_dependent_launch;
using lkd::mbar_arrive;
using lkd::mbar_expect_tx;
using lkd::mbar_init;
using lkd::mbar_try_wait;
using lkd::wait;
using lkd::smem_addr;
using lkd::wait_for_prerequisite_grid;

constexpr int kRows = 128;               // rows of a tile: M of the products, lanes of tensor memory
constexpr int kSoftWarps = 4;            // one thread per row
constexpr int kLoadWarp = 4, kMmaWarp = 5;
constexpr int kThreads = 192;
constexpr int kJoinWarps = 8, kJoinThreads = 32 * kJoinWarps;       // of a CTA of join_kernel
constexpr int kFewParts = 4;             // parts that a warp joins by itself (1: 512 items of 48 rows 265 us, not 255)
constexpr int kMaxSms = 160;             // the workspace is sized for this many (a GB300 has 152)
constexpr float kLazy = 8.0f;            // log2 of how far m may lag behind a row's maximum
// log2 of the factor that all weights (and so their sum) carry: float16's 2^-24 steps end
// that much further down, and 2^(kLazy + 7) is still in its range
template <typename T>
constexpr float kRaise = std::is_same<T, __half>::value ? 7.0f : 0.0f;
constexpr int kBarBytes = 1024;          // barriers and small state ahead of the tiles

// Shared memory and tensor memory of head size D.  A slot holds one tile of K, of V or of both.
template <int D>
struct Shape {
    static constexpr int kCtas = D == 256 ? 1 : 2;           // per SM
    // Positions of a tile.  The thread that issues the products takes 0.8 us a tile (four
    // waits, a dozen instructions of 40 ns); at D = 64 a tile of 64 positions has 16 KB,
    // for which that is too long (16 requests of 512 to 262144 positions, blocks of 8, 14
    // heads on 2: 97 us, and 79 in tiles of 128).  At D = 128 and 256 64 positions have 32
    // and 64 KB, and 128 would leave less than two tiles of K and V in a CTA's memory.
    static constexpr int kTile = D == 64 ? 128 : 64;
    // What an item's begin and end cost, in tiles.  2048 items of 1 to 2048 positions and 32
    // rows at D = 128 take 100, 90, 87, 94 us where it is counted as 2, 3, 4, 6 tiles; as many
    // of 56 rows at D = 64 99, 96, 95, 99 us, 512 of 32 rows at D = 256 69, 64, 61, 65.
    static constexpr int kItemUnits = 4;
    // D = 64: K and V share a slot (a wait and a commit less), and one S tile is enough,
    // since P has tensor memory of its own: the next S comes as soon as this one is read.
    // Otherwise two S tiles, P over S, and slots for K and V apart, which fill earlier.
    static constexpr bool kPair = D == 64, kOwnP = D == 64;
    static constexpr int kTileBytes = kTile * D * 2;         // of K or of V
    static constexpr int kSlotBytes = kPair ? 2 * kTileBytes : kTileBytes;
    static constexpr int kQBytes = kRows * D * 2;
    static constexpr int kSlots = D == 256 ? 5 : (112 * 1024 - kQBytes) / kSlotBytes;
    static constexpr int kSmem = kBarBytes + kQBytes + kSlots * kSlotBytes;
    static constexpr int kBufs = kOwnP ? 1 : 2;              // S tiles in flight
    static constexpr int kCols = D == 256 ? 512 : 256;       // tensor memory: S, P where it is apart, O
    static constexpr int kP = kOwnP ? kBufs * kTile : 0, kPStep = kOwnP ? kTile / 2 : kTile;
    static constexpr int kO = kOwnP ? kP + kBufs * kPStep : kBufs * kTile;
    static_assert(kO + D <= kCols, "tensor memory");
    static constexpr int kAhead = 1;                         // S products issued before the oldest P V
};

struct Meta {                            // one per CTA: the item it began and did not end
    int32_t r, h, mt, last;              // r = -1: none; last = the CTA that ended it
    int32_t rows, failed, pad[2];
};

struct Params {
    CUtensorMap k_map, v_map;
    const void *q;
    int64_t qb, qn, qh;
    const int32_t *table, *kv_len, *q_len;
    int32_t B, N, Hq, Hkv, G, max_pages, pages, page_shift, window, ctas, part_rows, cache_rows;
    float c;                             // |scale| * log2(e)
    int32_t negate;
    void *out;
    float *lse;
    Meta *meta;                          // [ctas]
    float *parts;                        // [2 * ctas]: O [part_rows][D], m [part_rows], sum [part_rows]
    uint64_t limit;                      // clocks that a wait may take
};

// ---------------------------------------------------------------- the work ----
// Request r's part of the work: tokens of the block, positions its rows see, tiles.
struct Request {
    int32_t n, kv;
    int32_t lo, end;                     // some row sees positions [lo, end)
    int32_t t0, nt, mts;                 // first tile, tiles, row tiles
};

template <typename S>
__device__ __noinline__ Request request_of(const Params &p, int r) {
    Request q;
    q.n = p.q_len ? min(max(p.q_len[r], 0), p.N) : p.N;
    q.kv = max(p.kv_len[r], 0);
    q.end = int32_t(min(int64_t(q.kv) + q.n, int64_t(p.max_pages) << p.page_shift));     // at most 2^31 - 129
    q.lo = p.window > 0 ? max(q.kv - p.window + 1, 0) : 0;
    if (q.n == 0 || q.end <= q.lo) {
        q.t0 = q.nt = 0;
    } else {
        q.t0 = q.lo / S::kTile;
        q.nt = (q.end + S::kTile - 1) / S::kTile - q.t0;
    }
    q.mts = (q.n * p.G + kRows - 1) / kRows;
    return q;
}

// Units: an item's tiles, after kItemUnits for its begin and end (its Q, its result), so
// that a CTA with many short items gets fewer tiles.
template <typename S>
__device__ inline int32_t item_units(const Request &q) {
    return q.nt ? q.nt + S::kItemUnits : 0;
}
template <typename S>
__device__ inline int64_t units_of(const Params &p, const Request &q) {
    return int64_t(p.Hkv) * q.mts * item_units<S>(q);
}

// A CTA's walk over its range of units, item by item; every role takes the same steps.
template <typename S>
struct Walk {
    int32_t r, h, mt;
    Request q;
    int32_t u;                           // this item's first unit in the range
    int32_t a, b;                        // its tiles [a, b) of [0, q.nt) are this CTA's; b = 0: none
    int64_t left;                        // units of the range not yet handed out, this item's excluded

    __device__ void start(const Params &p, int32_t r0, int64_t off, int64_t count) {
        r = r0;
        left = count;
        q = request_of<S>(p, r);
        a = b = 0;
        if (count <= 0) return;
        const int64_t item = off / item_units<S>(q);
        h = int32_t(item / q.mts);
        mt = int32_t(item % q.mts);
        u = int32_t(off - item * item_units<S>(q));
        take();
        if (b == 0) next(p);
    }
    __device__ void take() {
        const int64_t can = item_units<S>(q) - u;
        const int32_t n = int32_t(left < can ? left : can);
        a = max(u - S::kItemUnits, 0);
        b = max(u + n - S::kItemUnits, 0);
        left -= n;
    }
    __device__ bool valid() const { return b > 0; }
    __device__ void next(const Params &p) {
        do {
            a = b = 0;
            if (left <= 0) return;
            u = 0;
            if (++mt == q.mts) {
                mt = 0;
                if (++h == p.Hkv) {
                    h = 0;
                    do {                                 // left > 0: a later request has units
                        if (++r >= p.B) return;
                        q = request_of<S>(p, r);
                    } while (q.nt == 0);
                }
            }
            take();
        } while (b == 0);                                // the range ends before the item's first tile
    }
};

// ------------------------------------------------------------------ tcgen05 ----
__device__ inline void tc_alloc(uint32_t smem_out, uint32_t cols) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_out), "r"(cols) : "memory");
}
__device__ inline void tc_dealloc(uint32_t addr, uint32_t cols) {
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(addr), "r"(cols) : "memory");
}
__device__ inline void tc_relinquish() {
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
}
__device__ inline void tc_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ inline void tc_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ inline void tc_commit(uint32_t bar) {
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}

// D[tmem] (+)= A[smem] B[smem], and the same with A in tensor memory.
__device__ inline void tc_mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(uint32_t(accumulate))
        : "memory");
}
__device__ inline void tc_mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, bool accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
        "r"(a), "l"(b), "r"(idesc), "r"(uint32_t(accumulate))
        : "memory");
}
// The same into some of the warps' lanes only: bit w of `quads` set = lanes 32 w .. 32 w + 31.
__device__ inline void tc_mma_ts_quads(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, bool accumulate, uint32_t quads) {
    const uint32_t off0 = quads & 1 ? 0u : ~0u, off1 = quads & 2 ? 0u : ~0u;
    const uint32_t off2 = quads & 4 ? 0u : ~0u, off3 = quads & 8 ? 0u : ~0u;
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, {%5, %6, %7, %8}, p;\n\t}" ::"r"(d),
        "r"(a), "l"(b), "r"(idesc), "r"(uint32_t(accumulate)), "r"(off0), "r"(off1), "r"(off2), "r"(off3)
        : "memory");
}

// 32 or 16 columns of this warp's 32 lanes, and the wait that makes them usable; the
// stores of 32, 16 or 8.
__device__ inline void tc_ld(uint32_t addr, uint32_t (&r)[32]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
        "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
          "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
          "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(addr));
}
__device__ inline void tc_wait_ld(uint32_t (&r)[32]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                   "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]),
                   "+r"(r[15]), "+r"(r[16]), "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]),
                   "+r"(r[22]), "+r"(r[23]), "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]),
                   "+r"(r[29]), "+r"(r[30]), "+r"(r[31])::"memory");
}
__device__ inline void tc_st(uint32_t addr, const uint32_t (&r)[32]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%32], "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
        "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31};" ::"r"(r[0]),
        "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]),
        "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]),
        "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]),
        "r"(r[29]), "r"(r[30]), "r"(r[31]), "r"(addr)
        : "memory");
}
__device__ inline void tc_ld(uint32_t addr, uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(addr));
}
__device__ inline void tc_wait_ld(uint32_t (&r)[16]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                   "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]),
                   "+r"(r[15])::"memory");
}
__device__ inline void tc_st(uint32_t addr, const uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15};" ::"r"(r[0]),
        "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]),
        "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(addr)
        : "memory");
}
__device__ inline void tc_st(uint32_t addr, const uint32_t (&r)[8]) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%8], {%0,%1,%2,%3,%4,%5,%6,%7};" ::"r"(r[0]), "r"(r[1]),
                 "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(addr)
                 : "memory");
}
__device__ inline void tc_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// Shared-memory operand descriptor, 128-byte swizzle: start, leading and stride byte
// offsets in units of 16 bytes, version 1, layout 2.  K-major (Q, K): rows of 128
// bytes, groups of 8 rows `stride` apart.  MN-major (V): 64 columns per 128-byte row,
// groups of 8 rows `stride` apart, the next 64 columns `lead` away.
__device__ inline uint64_t operand_desc(uint32_t addr, uint32_t lead, uint32_t stride) {
    return uint64_t((addr >> 4) & 0x3fff) | (uint64_t((lead >> 4) & 0x3fff) << 16) |
           (uint64_t((stride >> 4) & 0x3fff) << 32) | (uint64_t(1) << 46) | (uint64_t(2) << 61);
}

// Instruction descriptor of kind::f16: float32 accumulator, A K-major, B K-major or
// (b_mn) MN-major, M = 128, N = n.
template <typename T>
__device__ constexpr uint32_t instr_desc(int n, bool b_mn);
template <>
__device__ constexpr uint32_t instr_desc<__half>(int n, bool b_mn) {
    return (1u << 4) | (uint32_t(b_mn) << 16) | (uint32_t(n / 8) << 17) | (uint32_t(kRows / 16) << 24);
}
template <>
__device__ constexpr uint32_t instr_desc<__nv_bfloat16>(int n, bool b_mn) {
    return instr_desc<__half>(n, b_mn) | (1u << 7) | (1u << 10);
}

__device__ inline void tma_load(uint32_t dst, const CUtensorMap *map, int32_t x, int32_t y, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4}], [%2];" ::"r"(dst),
        "l"(map), "r"(bar), "r"(x), "r"(y)
        : "memory");
}

__device__ inline void copy16(uint32_t dst, const void *src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}

__device__ inline float exp2_approx(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Two probabilities as one word of the type, the first in the low half.
__device__ inline uint32_t pack2(float lo, float hi, __half) {
    uint32_t d;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
    return d;
}
__device__ inline uint32_t pack2(float lo, float hi, __nv_bfloat16) {
    uint32_t d;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
    return d;
}

// ------------------------------------------------------------------- shared ----
// Ahead of the tiles: barriers (8 bytes each) and a few words.
struct Head {
    uint64_t full[16], empty[16];        // slots
    uint64_t s_full[3], p_ready[3], pv_done[3], q_ready, staged, sync, s_free, drain;
    uint32_t tmem, failed;
    int32_t start_r;
    int64_t start_off, total;
    int64_t warp_sum[kThreads / 32];
};
static_assert(sizeof(Head) <= kBarBytes, "Head fits ahead of the tiles");

// The same for a whole warp: every lane waits, and all go on or none does.
__device__ inline bool warp_wait(uint32_t bar, uint32_t parity, volatile uint32_t *failed, uint64_t limit) {
    return __all_sync(0xffffffffu, wait(bar, parity, failed, limit));
}

// A place in a ring of N and the parity of how often the ring has been round.
template <int N>
struct Place {
    uint32_t at, phase;
    __device__ void step(uint32_t by) {
        at += by;
        if (at >= N) {
            at -= N;
            phase ^= 1;
        }
    }
};

template <typename T, int D, int REP>
__global__ void __launch_bounds__(kThreads, Shape<D>::kCtas) attention_kernel(const __grid_constant__ Params p) {
    using S = Shape<D>;
    constexpr int kTile = S::kTile;
    extern __shared__ __align__(1024) unsigned char smem[];
    Head &hd = *reinterpret_cast<Head *>(smem);
    const uint32_t q_smem = smem_addr(smem) + kBarBytes;
    const uint32_t slots = q_smem + S::kQBytes;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, cta = blockIdx.x;
    volatile uint32_t *failed = &hd.failed;
    auto full = [&](int s) { return smem_addr(&hd.full[s]); };
    auto empty = [&](int s) { return smem_addr(&hd.empty[s]); };

    if (tid == 0) {
        for (int s = 0; s < S::kSlots; ++s) {
            mbar_init(full(s), 1);
            mbar_init(empty(s), 1);
        }
        for (int k = 0; k < S::kBufs; ++k) {
            mbar_init(smem_addr(&hd.s_full[k]), 1);
            mbar_init(smem_addr(&hd.p_ready[k]), kRows);
            mbar_init(smem_addr(&hd.pv_done[k]), 1);
        }
        mbar_init(smem_addr(&hd.q_ready), kRows);
        mbar_init(smem_addr(&hd.staged), kRows);
        mbar_init(smem_addr(&hd.sync), kRows);
        mbar_init(smem_addr(&hd.s_free), kRows);
        mbar_init(smem_addr(&hd.drain), 1);
        lkd::fence_barrier_init();
        hd.failed = 0;
    }
    if (warp == kMmaWarp) {
        tc_alloc(smem_addr(&hd.tmem), S::kCols);
        tc_relinquish();
    }
    wait_for_prerequisite_grid();
    allow_dependent_launch();

    // the range of this CTA: units [start, stop) of all requests' units end to end.  A
    // thread per request and a scan; more requests than threads take a second pass
    auto scan = [&](int64_t x) {                         // over the warp, its total to warp_sum
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int64_t y = __shfl_up_sync(0xffffffffu, x, d);
            if (lane >= d) x += y;
        }
        if (lane == 31) hd.warp_sum[warp] = x;
        return x;
    };
    int64_t own = 0;
    for (int r = tid; r < p.B; r += kThreads) own += units_of<S>(p, request_of<S>(p, r));
    int64_t upto = scan(own);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = hd.tmem;
    int64_t total = 0;
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) total += hd.warp_sum[w];
    const int64_t ctas = min(int64_t(p.ctas), total);    // with a range of their own
    const int64_t start = cta < ctas ? total * cta / ctas : total, stop = cta < ctas ? total * (cta + 1) / ctas : total;
    const int64_t count = stop - start;
    if (count > 0) {
        int64_t before = 0;                              // units of the requests ahead of this pass
        for (int r0 = 0; r0 < p.B && before <= start; r0 += kThreads) {
            const int r = r0 + tid;
            if (p.B > kThreads) {
                own = r < p.B ? units_of<S>(p, request_of<S>(p, r)) : 0;
                __syncthreads();                         // warp_sum's last readers are done
                upto = scan(own);
                __syncthreads();
            }
            int64_t ahead = before + upto - own;
            for (int w = 0; w < kThreads / 32; ++w) {
                if (w < warp) ahead += hd.warp_sum[w];
                before += hd.warp_sum[w];
            }
            if (ahead <= start && start < ahead + own) {
                hd.start_r = r;
                hd.start_off = start - ahead;
            }
        }
    }
    __syncthreads();

    Walk<S> wk;
    if (count > 0) wk.start(p, hd.start_r, hd.start_off, count);

    if (warp == kMmaWarp) {
        // rows of the block past q_len, and those of requests that see nothing (this warp
        // has time: Q takes 2 us to come)
        for (int r = cta; r < p.B; r += p.ctas) {
            const Request q = request_of<S>(p, r);
            const int64_t i0 = (int64_t(r) * p.N + (q.nt ? q.n : 0)) * p.Hq, i1 = int64_t(r + 1) * p.N * p.Hq;
            for (int64_t x = i0 * (D / 8) + lane; x < i1 * (D / 8); x += 32)
                reinterpret_cast<uint4 *>(p.out)[x] = make_uint4(0, 0, 0, 0);
            if (p.lse)
                for (int64_t x = i0 + lane; x < i1; x += 32) p.lse[x] = -INFINITY;
        }
    }
    if (count > 0 && warp == kLoadWarp) {
        // ---- loads: K and V of tile after tile, slot after slot ----
        const int box_rows = min(kTile, 1 << p.page_shift);
        const int per_tile = kTile / box_rows;           // pages of a tile (1 when a page holds whole tiles)
        const int boxes = per_tile * (D / 64);           // at most 8 * 4
        const int my_page = lane % per_tile, my_col = lane / per_tile;
        uint32_t n = 0;                                  // slots filled so far
        Place<S::kSlots> to{0, 0};                       // the next one
        bool ok = true;
        // page ids, 32 at a time, and the next 32 ahead of their use; the first of an item
        // are on their way during the item before
        auto entry = [&](int32_t r, int64_t at) { return at < p.max_pages ? p.table[int64_t(r) * p.max_pages + at] : -1; };
        auto first_page = [&](const Walk<S> &w) { return (int64_t(w.q.t0 + w.a) * kTile) >> p.page_shift; };
        Walk<S> ahead = wk;
        int32_t ids = wk.valid() ? entry(wk.r, first_page(wk) + lane) : -1;
        for (; ok && wk.valid(); wk = ahead) {
            int64_t base = first_page(wk);
            int32_t cur = ids, nxt = entry(wk.r, base + 32 + lane);
            for (int t = wk.a; ok && t < wk.b; ++t) {
                const int64_t x0 = int64_t(wk.q.t0 + t) * kTile;
                int64_t at = x0 >> p.page_shift;
                if (at - base >= 32) {                   // a tile's pages never straddle a window: 32 % per_tile == 0
                    base += 32;
                    cur = nxt;
                    nxt = entry(wk.r, base + 32 + lane);
                }
                const int32_t page = __shfl_sync(0xffffffffu, cur, int(at - base) + my_page);
                const int64_t x = x0 + my_page * box_rows;
                // a row past the map's end reads as zeros: absent pages, and pages past the end
                int32_t y = p.cache_rows;
                if (page >= 0 && page < p.pages && x < wk.q.end)
                    y = ((page * p.Hkv + wk.h) << p.page_shift) + int32_t(x & ((1 << p.page_shift) - 1));
#pragma unroll
                for (int part = 0; part < (S::kPair ? 1 : 2); ++part, ++n) {
                    const uint32_t s = to.at;
                    if (!warp_wait(empty(s), to.phase ^ 1, failed, p.limit)) {
                        ok = false;
                        break;
                    }
                    to.step(1);
                    if (lane == 0) mbar_expect_tx(full(s), S::kSlotBytes);
                    __syncwarp();
                    const uint32_t dst = slots + s * S::kSlotBytes + my_col * (kTile * 128) + my_page * box_rows * 128;
                    if (lane < boxes) {
                        tma_load(dst, part ? &p.v_map : &p.k_map, my_col * 64, y, full(s));
                        if (S::kPair) tma_load(dst + S::kTileBytes, &p.v_map, my_col * 64, y, full(s));
                    }
                }
                if (t == wk.a) {
                    ahead.next(p);
                    if (ahead.valid()) ids = entry(ahead.r, first_page(ahead) + lane);
                }
            }
        }
        {                                                // no copy outlives the CTA, whoever gave up
            const uint32_t in_flight = n < uint32_t(S::kSlots) ? n : uint32_t(S::kSlots);
            for (uint32_t k = n - in_flight; k < n; ++k) {
                const uint64_t until = lkd::global_ns() + 1000000000ull;
                while (!mbar_try_wait(full(k % S::kSlots), (k / S::kSlots) & 1) && lkd::global_ns() < until) {
                }
            }
        }
    } else if (count > 0 && warp == kMmaWarp) {
        // ---- products, by one thread ----
        if (lane == 0) {
            // (an instruction at a time: places and phases are carried along, and descriptors
            // differ in their low words only)
            constexpr uint32_t kQk = instr_desc<T>(kTile, false), kPv = instr_desc<T>(D, true);
            constexpr uint32_t kSlotStep = S::kSlotBytes / 16;
            const uint64_t q_desc = operand_desc(q_smem, 16, 1024), k_desc = operand_desc(slots, 16, 1024);
            const uint64_t v_desc = operand_desc(slots + (S::kPair ? S::kTileBytes : 0), kTile * 128, 1024);
            const uint32_t q_lo = uint32_t(q_desc), q_hi = uint32_t(q_desc >> 32);
            const uint32_t k_lo = uint32_t(k_desc), k_hi = uint32_t(k_desc >> 32);
            const uint32_t v_lo = uint32_t(v_desc), v_hi = uint32_t(v_desc >> 32);
            auto desc = [](uint32_t hi, uint32_t lo) { return (uint64_t(hi) << 32) | lo; };
            Place<S::kSlots> k_at{0, 0}, v_at{S::kPair ? 0u : 1u, 0};    // the next K and V slots
            Place<S::kBufs> s_at{0, 0}, p_at{0, 0};      // the next S tile to write, the next P to use
            uint32_t item = 0;
            bool ok = true, used = false;                // used: S tiles have been round once
            auto pv = [&](bool first) {                  // the next tile's P V into O
                ok = wait(smem_addr(&hd.p_ready[p_at.at]), p_at.phase, failed, p.limit) &&
                     (S::kPair || wait(full(v_at.at), v_at.phase, failed, p.limit));
                if (!ok) return;
                tc_fence_after();
                const uint32_t lo = v_lo + v_at.at * kSlotStep, a = tmem + S::kP + p_at.at * S::kPStep;
#pragma unroll
                for (int j = 0; j < kTile / 16; ++j) {
                    if (REP == 1) {
                        tc_mma_ts(tmem + S::kO, a + j * 8, desc(v_hi, lo + j * 128), kPv, !(first && j == 0));
                    } else {                             // these 16 positions: into their copy's lanes
                        constexpr int kSteps = kTile / 16 / REP, kQuads = kSoftWarps / REP;
                        tc_mma_ts_quads(tmem + S::kO, a + j * 8, desc(v_hi, lo + j * 128), kPv,
                                        !(first && j % kSteps == 0), ((1u << kQuads) - 1) << (j / kSteps * kQuads));
                    }
                }
                tc_commit(empty(v_at.at));
                tc_commit(smem_addr(&hd.pv_done[p_at.at]));
                v_at.step(S::kPair ? 1 : 2);
                p_at.step(1);
            };
            for (; ok && wk.valid(); wk.next(p), ++item) {
                ok = wait(smem_addr(&hd.q_ready), item & 1, failed, p.limit);
                for (int t = wk.a; ok && t < wk.b + S::kAhead; ++t) {
                    if (t < wk.b) {
                        // K is there, and the S of kBufs tiles ago has been read; where P lies over S,
                        // its product is over too
                        ok = wait(full(k_at.at), k_at.phase, failed, p.limit) &&
                             (!used || wait(S::kOwnP ? smem_addr(&hd.s_free) : smem_addr(&hd.pv_done[s_at.at]),
                                            s_at.phase ^ 1, failed, p.limit));
                        if (!ok) break;
                        tc_fence_after();
                        const uint32_t lo = k_lo + k_at.at * kSlotStep, d = tmem + s_at.at * kTile;
#pragma unroll
                        for (int j = 0; j < D / 16; ++j)
                            tc_mma_ss(d, desc(q_hi, q_lo + (j / 4) * (kRows * 8) + (j % 4) * 2),
                                      desc(k_hi, lo + (j / 4) * (kTile * 8) + (j % 4) * 2), kQk, j > 0);
                        if (!S::kPair) tc_commit(empty(k_at.at));
                        tc_commit(smem_addr(&hd.s_full[s_at.at]));
                        k_at.step(S::kPair ? 1 : 2);
                        s_at.step(1);
                        used = used || s_at.phase;
                    }
                    if (ok && t - wk.a >= S::kAhead) pv(t - S::kAhead == wk.a);
                }
            }
            {                                            // nor does a product
                tc_commit(smem_addr(&hd.drain));
                const uint64_t until = lkd::global_ns() + 1000000000ull;
                while (!mbar_try_wait(smem_addr(&hd.drain), 0) && lkd::global_ns() < until) {
                }
            }
        }
        __syncwarp();
    } else if (warp < kSoftWarps) {
        // ---- softmax: a thread per row, or REP threads in as many warps, each for its
        // kCols columns of every tile ----
        constexpr int kQuads = kSoftWarps / REP, kCols = kTile / REP;    // warps of a copy; columns of a thread
        const uint32_t lanes = uint32_t(warp * 32) << 16;
        const int copy = warp / kQuads, col0 = copy * kCols;
        const int row = (warp % kQuads) * 32 + lane, thread = warp * 32 + lane;
        uint32_t it = 0, item = 0, syncs = 0;
        Place<S::kBufs> s_at{0, 0}, before{0, 0};        // this tile's S, and the last tile's
        // all the threads here, false on failure
        auto soft_sync = [&]() {
            mbar_arrive(smem_addr(&hd.sync));
            return warp_wait(smem_addr(&hd.sync), syncs++ & 1, failed, p.limit);
        };
        unsigned char *stage = smem + kBarBytes + warp * 4096;       // 32 rows of 128 bytes, in Q's place
        Meta meta{-1, 0, 0, 0, 0, 0, {0, 0}};
        bool ok = true;
        // Q: a thread's pieces of 16 bytes.  Where they are few, the next item's are on their
        // way during this one; otherwise, and where registers are short (two copies at D = 64:
        // 95 us without, 99 with), they go from global to shared memory by themselves.
        constexpr int kCh = D / 8, kStep = kRows / kCh;  // pieces of a row, rows of a pass
        constexpr int kLoads = kRows / REP / kStep;
        constexpr bool kEarly = kLoads <= 4 && !(D == 64 && REP == 2);
        const int ch = thread % kCh;
        auto q_piece = [&](const Walk<S> &w, int y) {
            const uint32_t ry = w.mt * kRows + y, iy = ry / uint32_t(p.G);
            return static_cast<const T *>(p.q) + w.r * p.qb + w.h * p.G * p.qh + ch * 8 + iy * p.qn +
                   (ry - iy * p.G) * p.qh;
        };
        uint4 early[kEarly ? kLoads : 1];
        auto load_q = [&](const Walk<S> &w) {
            const int rows = min(kRows, w.q.n * p.G - w.mt * kRows);
#pragma unroll
            for (int k = 0; k < (kEarly ? kLoads : 0); ++k) {
                const int y = thread / kCh + k * kStep;
                if (y < rows) early[k] = *reinterpret_cast<const uint4 *>(q_piece(w, y));
            }
        };
        Walk<S> ahead = wk;
        auto advance = [&]() {
            if (kEarly) wk = ahead;
            else wk.next(p);
        };
        if (count > 0 && wk.valid()) load_q(wk);
        for (; count > 0 && ok && wk.valid(); advance(), ++item) {
            const Request &q = wk.q;
            const int rows = min(kRows, q.n * p.G - wk.mt * kRows);
            const int rr = wk.mt * kRows + row;          // row of the request: token, then head of the group
            const bool live = row < rows;
            const int i = live ? rr / p.G : 0;
            const int head = wk.h * p.G + (live ? rr - i * p.G : 0);
            // Q where the products' swizzle wants it (idle rows keep what was there: a row of S
            // depends on its own row of Q only).  Before it, the last item's result has left
            // these bytes.
            if (item > 0 && !warp_wait(smem_addr(&hd.staged), (item - 1) & 1, failed, p.limit)) {
                ok = false;
                break;
            }
            {
                const uint32_t flip = p.negate ? 0x80008000u : 0u;
                unsigned char *dst = smem + kBarBytes + (ch >> 3) * (kRows * 128);
                auto at = [&](int y, int k) { return dst + (y + k * kQuads * 32) * 128 + (((ch & 7) ^ (y & 7)) << 4); };
                if (kEarly) {
#pragma unroll
                    for (int k = 0; k < kLoads; ++k) {
                        const int y = thread / kCh + k * kStep;
                        const uint4 v = early[k];
                        if (y < rows)
#pragma unroll
                            for (int c = 0; c < REP; ++c)
                                *reinterpret_cast<uint4 *>(at(y, c)) =
                                    make_uint4(v.x ^ flip, v.y ^ flip, v.z ^ flip, v.w ^ flip);
                    }
                } else {
                    for (int y = thread / kCh; y < rows; y += kStep)
#pragma unroll
                        for (int c = 0; c < REP; ++c) copy16(smem_addr(at(y, c)), q_piece(wk, y));
                    asm volatile("cp.async.wait_all;" ::: "memory");
                    if (flip)
                        for (int y = thread / kCh; y < rows; y += kStep)
#pragma unroll
                            for (int c = 0; c < REP; ++c) {
                                uint4 *v = reinterpret_cast<uint4 *>(at(y, c));
                                *v = make_uint4(v->x ^ flip, v->y ^ flip, v->z ^ flip, v->w ^ flip);
                            }
                }
                lkd::fence_proxy_async_smem();
                mbar_arrive(smem_addr(&hd.q_ready));
            }
            if (kEarly) {
                ahead.next(p);
                if (ahead.valid()) load_q(ahead);
            }
            // positions this row sees: [see0, see1)
            const int64_t pos = int64_t(q.kv) + i;
            const int64_t see1 = min(pos + 1, int64_t(q.end));
            const int64_t see0 = p.window > 0 ? max(pos - p.window + 1, int64_t(0)) : 0;
            float m = -INFINITY, sum = 0.0f;             // m: the raw product the sums are relative to
            const bool warp_live = (warp % kQuads) * 32 < rows;
            for (int t = wk.a; t < wk.b; ++t, ++it) {
                const int64_t x0 = int64_t(q.t0 + t) * kTile;
                const uint32_t buf = s_at.at;
                if (!warp_wait(smem_addr(&hd.s_full[buf]), s_at.phase, failed, p.limit)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                if (x0 < q.lo || x0 + kTile > q.end) {
                    // rows of V that no row of the block sees may hold anything: zeros
                    const uint32_t n = S::kPair ? it : 2 * it + 1;
                    const int s = n % S::kSlots;
                    if (!warp_wait(full(s), (n / S::kSlots) & 1, failed, p.limit)) {
                        ok = false;
                        break;
                    }
                    unsigned char *v = smem + kBarBytes + S::kQBytes + s * S::kSlotBytes + (S::kPair ? S::kTileBytes : 0);
                    for (int x = thread; x < kTile * (D / 8); x += kRows) {
                        const int y = (x >> 3) & (kTile - 1);
                        if (x0 + y < q.lo || x0 + y >= q.end)
                            *reinterpret_cast<uint4 *>(v + x * 16) = make_uint4(0, 0, 0, 0);
                    }
                    lkd::fence_proxy_async_smem();
                }
                const bool fresh = t == wk.a;
                if (warp_live) {
                    // a thread's columns, 32 (or its 16) at a time; 64 stay in registers, 128 are
                    // read twice, for the maximum and for the weights
                    constexpr int kStep = kCols < 32 ? kCols : 32, kSteps = kCols / kStep;
                    constexpr bool kTwice = kCols > 64;
                    constexpr int kUnroll = kTwice ? 1 : kSteps;
                    const uint32_t at = tmem + lanes + buf * kTile + col0;
                    uint32_t r[kTwice ? 1 : kSteps][kStep];
                    // tiles that some row of the request sees less than all of
                    const bool masked = x0 + kTile > min(int64_t(q.kv) + 1, int64_t(q.end)) ||
                                        (p.window > 0 && x0 < int64_t(q.kv) + q.n - p.window);
                    const int c0 = int(min(max(see0 - x0, int64_t(0)), int64_t(kTile))) - col0;
                    const int c1 = int(min(max(see1 - x0, int64_t(0)), int64_t(kTile))) - col0;
                    auto hide = [&](uint32_t (&x)[kStep], int from) {
                        if (!masked) return;
#pragma unroll
                        for (int j = 0; j < kStep; ++j)
                            if (from + j < c0 || from + j >= c1) x[j] = 0xff800000u;
                    };
                    float mx = -INFINITY;
                    if (!kTwice) {
#pragma unroll
                        for (int h = 0; h < kSteps; ++h) tc_ld(at + h * kStep, r[kTwice ? 0 : h]);
#pragma unroll
                        for (int h = 0; h < kSteps; ++h) tc_wait_ld(r[kTwice ? 0 : h]);
                        if (S::kOwnP) {                  // S is in registers: the next may come
                            tc_fence_before();
                            mbar_arrive(smem_addr(&hd.s_free));
                        }
                    }
#pragma unroll kUnroll
                    for (int h = 0; h < kSteps; ++h) {
                        uint32_t (&x)[kStep] = r[kTwice ? 0 : h];
                        if (kTwice) {
                            tc_ld(at + h * kStep, x);
                            tc_wait_ld(x);
                        }
                        hide(x, h * kStep);
#pragma unroll
                        for (int j = 0; j < kStep; j += 2)
                            mx = fmaxf(mx, fmaxf(__uint_as_float(x[j]), __uint_as_float(x[j + 1])));
                    }
                    const bool lift = mx > m && (fresh || m == -INFINITY || (mx - m) * p.c > kLazy);
                    // the last product is over: before O is brought to a new m, and before P is
                    // overwritten where there is one
                    if ((S::kOwnP && it > 0) || (!fresh && __any_sync(0xffffffffu, lift))) {
                        if (!warp_wait(smem_addr(&hd.pv_done[before.at]), before.phase, failed, p.limit)) {
                            ok = false;
                            break;
                        }
                        tc_fence_after();
                    }
                    if (fresh) {
                        m = mx;
                    } else if (__any_sync(0xffffffffu, lift)) {
                        const float f = !lift ? 1.0f : (m == -INFINITY ? 0.0f : exp2_approx((m - mx) * p.c));
                        if (lift) m = mx;
                        sum *= f;
#pragma unroll 1
                        for (int j = 0; j < D; j += 32) {
                            uint32_t o[32];
                            tc_ld(tmem + lanes + S::kO + j, o);
                            tc_wait_ld(o);
#pragma unroll
                            for (int k = 0; k < 32; ++k)
                                o[k] = __float_as_uint(f == 0.0f ? 0.0f : __uint_as_float(o[k]) * f);
                            tc_st(tmem + lanes + S::kO + j, o);
                        }
                    }
                    const float base = kRaise<T> - (m == -INFINITY ? 0.0f : m * p.c);
                    float part_sum[4] = {};
                    const uint32_t to = tmem + lanes + S::kP + buf * S::kPStep + copy * (kCols / 2);
                    uint32_t w[kTwice ? kStep / 2 : kCols / 2];
#pragma unroll kUnroll
                    for (int h = 0; h < kSteps; ++h) {
                        uint32_t (&x)[kStep] = r[kTwice ? 0 : h];
                        if (kTwice) {
                            tc_ld(at + h * kStep, x);
                            tc_wait_ld(x);
                            if (h == kSteps - 1 && S::kOwnP) {
                                tc_fence_before();
                                mbar_arrive(smem_addr(&hd.s_free));
                            }
                            hide(x, h * kStep);
                        }
#pragma unroll
                        for (int j = 0; j < kStep; j += 2) {
                            float a0 = exp2_approx(fmaf(__uint_as_float(x[j]), p.c, base));
                            float a1 = exp2_approx(fmaf(__uint_as_float(x[j + 1]), p.c, base));
                            if (masked) {                // also where c is 0
                                a0 = x[j] == 0xff800000u ? 0.0f : a0;
                                a1 = x[j + 1] == 0xff800000u ? 0.0f : a1;
                            }
                            part_sum[j & 2] += a0;
                            part_sum[(j & 2) + 1] += a1;
                            w[(kTwice ? 0 : h * kStep / 2) + j / 2] = pack2(a0, a1, T());
                        }
                        if (kTwice) tc_st(to + h * (kStep / 2), w);
                    }
                    sum += (part_sum[0] + part_sum[1]) + (part_sum[2] + part_sum[3]);
                    if (!kTwice) tc_st(to, w);
                    tc_wait_st();
                } else if (S::kOwnP) {
                    // an idle warp keeps step with the others: with one P tile, it would otherwise
                    // say that the next P is ready while this one is being written
                    mbar_arrive(smem_addr(&hd.s_free));
                    if (it > 0 && !warp_wait(smem_addr(&hd.pv_done[before.at]), before.phase, failed, p.limit)) {
                        ok = false;
                        break;
                    }
                }
                tc_fence_before();
                mbar_arrive(smem_addr(&hd.p_ready[buf]));
                before = s_at;
                s_at.step(1);
            }
            if (!ok) break;
            // the item's end: its rows, or this CTA's part of them.  Each thread has a row; 128
            // bytes of every row of the warp at a time go through shared memory, in Q's place
            // (the last S is there, so Q has been read; 16-byte pieces swizzled by the row), so
            // that whole lines are written.
            const bool whole = wk.a == 0 && wk.b == q.nt;
            const int my_row = lane >> 3, my_piece = lane & 7;       // of four rows at a time
            float f = 0.0f, all = 0.0f, big = -INFINITY;
            if (REP > 1) {
                // the copies' sums are added, each at the largest of their m: their factors, while
                // the last product runs
                float *own = reinterpret_cast<float *>(stage);
                own[lane] = m;
                own[32 + lane] = sum;
                if (!(ok = soft_sync())) break;
                const float *first = reinterpret_cast<const float *>(smem + kBarBytes + (warp % kQuads) * 4096);
#pragma unroll
                for (int k = 0; k < REP; ++k)
                    if (first[k * kQuads * 1024 + 32 + lane] != 0.0f) big = fmaxf(big, first[k * kQuads * 1024 + lane]);
#pragma unroll
                for (int k = 0; k < REP; ++k) {
                    const float mk = first[k * kQuads * 1024 + lane], sk = first[k * kQuads * 1024 + 32 + lane];
                    const float w = sk == 0.0f ? 0.0f : mk == big ? 1.0f : exp2_approx((mk - big) * p.c);
                    if (w != 0.0f) all += w * sk;
                    if (k == copy) f = w;
                }
                if (!(ok = soft_sync())) break;
                if (whole) f = all == 0.0f ? 0.0f : f / all;
            }
            if (!warp_wait(smem_addr(&hd.pv_done[before.at]), before.phase, failed, p.limit)) {
                ok = false;
                break;
            }
            tc_fence_after();
            // slot 2c + 1: the item began here; 2c: it began in an earlier range
            const int slot = 2 * cta + (wk.a == 0 ? 1 : 0);
            float *ws = p.parts + int64_t(slot) * (D + 2) * p.part_rows;
            if (REP > 1) {
                // every copy adds a part of the rows; Q's place holds half of the columns
                constexpr int kStrips = D / 64;          // of 32 columns, 16 KB each
#pragma unroll 1
                for (int j0 = 0; j0 < D; j0 += 32 * kStrips) {
                    if (j0 > 0 && !(ok = soft_sync())) break;
                    if (warp_live) {
#pragma unroll 1
                        for (int y = 0; y < kStrips; ++y) {
                            uint32_t o[32];
                            tc_ld(tmem + lanes + S::kO + j0 + 32 * y, o);
                            tc_wait_ld(o);
#pragma unroll
                            for (int k = 0; k < 8; ++k) {
                                uint32_t v[4];
#pragma unroll
                                for (int e = 0; e < 4; ++e)
                                    v[e] = f == 0.0f ? 0u : __float_as_uint(__uint_as_float(o[4 * k + e]) * f);
                                *reinterpret_cast<uint4 *>(stage + y * (kRows * 128) + lane * 128 +
                                                           ((k ^ (lane & 7)) << 4)) =
                                    make_uint4(v[0], v[1], v[2], v[3]);
                            }
                        }
                    }
                    if (!(ok = soft_sync())) break;
#pragma unroll 1
                    for (int t = 0; t < 32 / REP; t += 4) {
                        const int y = copy * (32 / REP) + t + my_row, full_y = (warp % kQuads) * 32 + y;
                        if (full_y < rows) {
                            const uint32_t ry = wk.mt * kRows + full_y, iy = ry / uint32_t(p.G);
                            const int64_t o_row =
                                (int64_t(wk.r) * p.N + iy) * p.Hq + wk.h * p.G + (ry - iy * uint32_t(p.G));
#pragma unroll 1
                            for (int strip = 0; strip < kStrips; ++strip) {
                                float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
                                for (int k = 0; k < REP; ++k) {
                                    const float4 u = *reinterpret_cast<const float4 *>(
                                        smem + kBarBytes + strip * (kRows * 128) + (warp % kQuads + k * kQuads) * 4096 +
                                        y * 128 + ((my_piece ^ (y & 7)) << 4));
                                    v.x += u.x;
                                    v.y += u.y;
                                    v.z += u.z;
                                    v.w += u.w;
                                }
                                const int at = j0 + 32 * strip + my_piece * 4;
                                if (whole)
                                    *reinterpret_cast<uint2 *>(static_cast<T *>(p.out) + o_row * D + at) =
                                        make_uint2(pack2(v.x, v.y, T()), pack2(v.z, v.w, T()));
                                else
                                    *reinterpret_cast<float4 *>(ws + full_y * D + at) = v;
                            }
                        }
                    }
                }
                if (!ok) break;
                if (live && copy == 0) {
                    if (!whole) {
                        ws[D * p.part_rows + row] = big;
                        ws[(D + 1) * p.part_rows + row] = all;
                    } else if (p.lse) {
                        p.lse[(int64_t(wk.r) * p.N + i) * p.Hq + head] =
                            all == 0.0f ? -INFINITY : 0.6931471805599453f * (big * p.c + (log2f(all) - kRaise<T>));
                    }
                }
            } else if (whole) {
                const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
                if (warp_live) {
#pragma unroll 1
                    for (int j = 0; j < D; j += 64) {
#pragma unroll 1
                        for (int half = 0; half < 2; ++half) {
                            uint32_t o[32];
                            tc_ld(tmem + lanes + S::kO + j + 32 * half, o);
                            tc_wait_ld(o);
#pragma unroll
                            for (int k = 0; k < 4; ++k) {
                                uint32_t w[4];
#pragma unroll
                                for (int e = 0; e < 4; ++e)          // (a row that sees nothing is 0)
                                    w[e] = sum == 0.0f ? 0u
                                                       : pack2(__uint_as_float(o[8 * k + 2 * e]) * inv,
                                                               __uint_as_float(o[8 * k + 2 * e + 1]) * inv, T());
                                *reinterpret_cast<uint4 *>(stage + lane * 128 + (((4 * half + k) ^ (lane & 7)) << 4)) =
                                    make_uint4(w[0], w[1], w[2], w[3]);
                            }
                        }
                        __syncwarp();
#pragma unroll
                        for (int t = 0; t < 32; t += 4) {
                            const int y = t + my_row;
                            if (warp * 32 + y < rows) {
                                const uint32_t ry = wk.mt * kRows + warp * 32 + y, iy = ry / uint32_t(p.G);
                                const int64_t o_row =
                                    (int64_t(wk.r) * p.N + iy) * p.Hq + wk.h * p.G + (ry - iy * uint32_t(p.G));
                                *reinterpret_cast<uint4 *>(static_cast<T *>(p.out) + o_row * D + j + my_piece * 8) =
                                    *reinterpret_cast<const uint4 *>(stage + y * 128 + ((my_piece ^ (y & 7)) << 4));
                            }
                        }
                        __syncwarp();
                    }
                    if (live && p.lse)
                        p.lse[(int64_t(wk.r) * p.N + i) * p.Hq + head] =
                            sum == 0.0f ? -INFINITY : 0.6931471805599453f * (m * p.c + (log2f(sum) - kRaise<T>));
                }
            } else {
                if (warp_live) {
#pragma unroll 1
                    for (int j = 0; j < D; j += 32) {
                        uint32_t o[32];
                        tc_ld(tmem + lanes + S::kO + j, o);
                        tc_wait_ld(o);
#pragma unroll
                        for (int k = 0; k < 8; ++k)
                            *reinterpret_cast<uint4 *>(stage + lane * 128 + ((k ^ (lane & 7)) << 4)) =
                                make_uint4(o[4 * k], o[4 * k + 1], o[4 * k + 2], o[4 * k + 3]);
                        __syncwarp();
#pragma unroll
                        for (int t = 0; t < 32; t += 4) {
                            const int y = (warp % kQuads) * 32 + t + my_row;
                            if (y < rows)
                                *reinterpret_cast<uint4 *>(ws + y * D + j + my_piece * 4) =
                                    *reinterpret_cast<const uint4 *>(stage + (t + my_row) * 128 +
                                                                     ((my_piece ^ ((t + my_row) & 7)) << 4));
                        }
                        __syncwarp();
                    }
                    if (live) {
                        ws[D * p.part_rows + row] = m;
                        ws[(D + 1) * p.part_rows + row] = sum;
                    }
                }
            }
            if (!whole) {
                if (wk.a == 0) {
                    // the CTA that has the item's last unit: the largest c whose range starts at or before it
                    const int64_t end = stop + (q.nt - wk.b);            // of the item's units
                    int64_t last = (end - 1) * ctas / total;
                    while (last + 1 < ctas && total * (last + 1) / ctas <= end - 1) ++last;
                    while (total * last / ctas > end - 1) --last;
                    meta = Meta{wk.r, wk.h, wk.mt, int32_t(last), rows, 0, {0, 0}};
                }
            }
            tc_fence_before();                           // O is read before the next item's products (p_ready)
            mbar_arrive(smem_addr(&hd.staged));
        }
        if (thread == 0) {
            meta.failed = ok ? 0 : 1;
            p.meta[cta] = meta;
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == kMmaWarp) tc_dealloc(tmem, S::kCols);
    // a wait that ran out in a role that does not write the record
    if (tid == 0 && hd.failed) p.meta[cta].failed = 1;
}

template <int D, int ROWS>
struct JoinSmem {
    static constexpr int kMost = kMaxSms * Shape<D>::kCtas;          // ranges at most
    float weights[ROWS][kMost], big[ROWS], sum[ROWS];
    float sums[kJoinWarps][ROWS][D];
    Meta metas[kMost];
};

// Joins the parts of the item that CTA c of attention_kernel began and did not end, the
// rows of this CTA's blockIdx.y.  Few parts (many items, each cut once or twice): a warp
// for two rows, the parts' maxima, sums and rows loaded together.  Many (few long items):
// ROWS rows at a time, first their weights 2^(c (m_k - M)), a warp per row and a lane
// per part; then each warp sums every eighth part over those rows, and the warps' sums
// are added.
template <typename T, int D, int ROWS>
__device__ void join_item(const Params &p, int c, const Meta &meta, JoinSmem<D, ROWS> &sm) {
    constexpr int E = D / 32;                            // columns of a lane
    constexpr int kFirst = 512 / D / ROWS > 0 ? 512 / D / ROWS * (D == 256 ? 1 : 2) : 1;     // parts of a warp in flight
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t size = int64_t(D + 2) * p.part_rows;   // of a part
    const int count = meta.last - c + 1;                 // the slot 2c + 1, then every second one after 2c + 2
    auto part = [&](int k) { return p.parts + int64_t(k ? 2 * (c + k) : 2 * c + 1) * size; };
    auto place = [&](int row) {                          // the row's place in out / D and in lse
        const int rr = meta.mt * kRows + row, i = rr / p.G;
        return (int64_t(meta.r) * p.N + i) * p.Hq + meta.h * p.G + (rr - i * p.G);
    };
    auto finish = [&](int row, const float (&o)[E], float big, float sum) {          // a warp's row
        const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
        uint32_t *dst = reinterpret_cast<uint32_t *>(static_cast<T *>(p.out) + place(row) * D + lane * E);
#pragma unroll
        for (int e = 0; e < E / 2; ++e) dst[e] = sum == 0.0f ? 0u : pack2(o[2 * e] * inv, o[2 * e + 1] * inv, T());
        if (lane == 0 && p.lse)
            p.lse[place(row)] = sum == 0.0f ? -INFINITY : 0.6931471805599453f * (big * p.c + (log2f(sum) - kRaise<T>));
    };
    if (count <= kFewParts) {
        constexpr int kPair = D == 256 ? 1 : 2;          // rows at a time
        const int step = gridDim.y * kJoinWarps;
        for (int row0 = blockIdx.y * kJoinWarps + warp; row0 < meta.rows; row0 += kPair * step) {
            float m[kPair][kFewParts], s[kPair][kFewParts];
            float2 v[kPair][kFewParts][E / 2];
#pragma unroll
            for (int y = 0; y < kPair; ++y)
#pragma unroll
                for (int k = 0; k < kFewParts; ++k) {
                    const int row = min(row0 + y * step, meta.rows - 1);
                    const float *src = part(k < count ? k : 0);
                    m[y][k] = k < count ? src[D * p.part_rows + row] : -INFINITY;
                    s[y][k] = k < count ? src[(D + 1) * p.part_rows + row] : 0.0f;   // 0: the row sees nothing of it
#pragma unroll
                    for (int e = 0; e < E / 2; ++e)
                        v[y][k][e] = reinterpret_cast<const float2 *>(src + row * D + lane * E)[e];
                }
#pragma unroll
            for (int y = 0; y < kPair; ++y) {
                if (row0 + y * step >= meta.rows) break;
                float big = -INFINITY, sum = 0.0f, o[E] = {};
#pragma unroll
                for (int k = 0; k < kFewParts; ++k)
                    if (s[y][k] != 0.0f) big = fmaxf(big, m[y][k]);
#pragma unroll
                for (int k = 0; k < kFewParts; ++k) {
                    const float w = s[y][k] == 0.0f ? 0.0f : m[y][k] == big ? 1.0f : exp2f((m[y][k] - big) * p.c);
                    if (w == 0.0f) continue;
                    sum += w * s[y][k];
#pragma unroll
                    for (int e = 0; e < E / 2; ++e) {
                        o[2 * e] += w * v[y][k][e].x;
                        o[2 * e + 1] += w * v[y][k][e].y;
                    }
                }
                finish(row0 + y * step, o, big, sum);
            }
        }
        return;
    }
    for (int row0 = blockIdx.y * ROWS; row0 < meta.rows; row0 += gridDim.y * ROWS) {
        const int rows = min(ROWS, meta.rows - row0);
        // the warp's first parts on their way while the weights are worked out
        float2 v[kFirst][ROWS][E / 2];
        auto fetch = [&](float2 (&to)[ROWS][E / 2], int k) {
            const float2 *src = reinterpret_cast<const float2 *>(part(k) + row0 * D + lane * E);
#pragma unroll
            for (int y = 0; y < ROWS; ++y)
#pragma unroll
                for (int e = 0; e < E / 2; ++e)
                    to[y][e] = k < count && y < rows ? src[y * (D / 2) + e] : make_float2(0.0f, 0.0f);
        };
#pragma unroll
        for (int f = 0; f < kFirst; ++f) fetch(v[f], warp + f * kJoinWarps);
        if (warp < rows) {
            const int row = row0 + warp;
            float *weight = sm.weights[warp];
            float big = -INFINITY, sum = 0.0f;
            for (int k = lane; k < count; k += 32) {
                const float mk = part(k)[D * p.part_rows + row], sk = part(k)[(D + 1) * p.part_rows + row];
                weight[k] = sk == 0.0f ? -INFINITY : mk;
                if (sk != 0.0f) big = fmaxf(big, mk);
            }
#pragma unroll
            for (int d = 16; d; d >>= 1) big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, d));
            for (int k = lane; k < count; k += 32) {
                const float mk = weight[k];
                const float w = mk == -INFINITY ? 0.0f : exp2f((mk - big) * p.c);
                weight[k] = w;
                if (w != 0.0f) sum += w * part(k)[(D + 1) * p.part_rows + row];
            }
#pragma unroll
            for (int d = 16; d; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
            if (lane == 0) {
                sm.big[warp] = big;
                sm.sum[warp] = sum;
            }
        }
        __syncthreads();
        float o[ROWS][E] = {};
        for (int k = warp; k < count; k += kFirst * kJoinWarps) {
#pragma unroll
            for (int f = 0; f < kFirst; ++f) {
                const int at = k + f * kJoinWarps;
                if (at >= count) break;
#pragma unroll
                for (int y = 0; y < ROWS; ++y) {
                    const float w = y < rows ? sm.weights[y][at] : 0.0f;
#pragma unroll
                    for (int e = 0; e < E / 2; ++e) {
                        o[y][2 * e] += w == 0.0f ? 0.0f : w * v[f][y][e].x;
                        o[y][2 * e + 1] += w == 0.0f ? 0.0f : w * v[f][y][e].y;
                    }
                }
            }
#pragma unroll
            for (int f = 0; f < kFirst; ++f) fetch(v[f], k + (kFirst + f) * kJoinWarps);
        }
        // the warps' sums; then warp y adds and finishes row y
#pragma unroll
        for (int y = 0; y < ROWS; ++y)
#pragma unroll
            for (int e = 0; e < E; ++e) sm.sums[warp][y][e * 32 + lane] = o[y][e];
        __syncthreads();
        if (warp < rows) {
            float all[E] = {};
#pragma unroll
            for (int w = 0; w < kJoinWarps; ++w)
#pragma unroll
                for (int e = 0; e < E; ++e) all[e] += sm.sums[w][warp][e * 32 + lane];
            finish(row0 + warp, all, sm.big[warp], sm.sum[warp]);
        }
        __syncthreads();                                 // shared memory has been read
    }
}

// The items that were cut: CTA x takes those begun by CTAs x, x + gridDim.x, ... of
// attention_kernel.  A wait that ran out anywhere makes the whole call's rows NaN.
template <typename T, int D, int ROWS>
__global__ void __launch_bounds__(kJoinThreads, D == 256 ? 2 : 3) join_kernel(const __grid_constant__ Params p) {
    __shared__ JoinSmem<D, ROWS> sm;
    wait_for_prerequisite_grid();
    allow_dependent_launch();
    const int tid = threadIdx.x;
    int bad = 0;
    for (int k = tid; k < p.ctas; k += kJoinThreads) {
        const Meta meta = p.meta[k];
        bad |= meta.failed;
        if (k % gridDim.x == blockIdx.x) sm.metas[k / gridDim.x] = meta;
    }
    if (__syncthreads_or(bad)) {
        const int64_t rows = int64_t(p.B) * p.N * p.Hq;
        const int64_t first = (int64_t(blockIdx.y) * gridDim.x + blockIdx.x) * kJoinThreads + tid;
        const int64_t step = int64_t(gridDim.x) * gridDim.y * kJoinThreads;
        for (int64_t x = first; x < rows * D; x += step) static_cast<T *>(p.out)[x] = T(NAN);
        if (p.lse)
            for (int64_t x = first; x < rows; x += step) p.lse[x] = NAN;
        return;
    }
    for (int c = blockIdx.x, k = 0; c < p.ctas; c += gridDim.x, ++k)
        if (sm.metas[k].r >= 0) join_item<T, D, ROWS>(p, c, sm.metas[k], sm);
}

// -------------------------------------------------------------------- host ----
int cuda_fail(cudaError_t e, const char *what) { return lookup_record_cuda_error(e, what); }

// CTAs of a call: as many as run at once on the device.
int ctas_for(int D, int sms) { return sms * (D == 256 ? 1 : 2); }

// Rows of a part: even, so that every part's rows are 16-byte aligned.
int part_rows_for(int64_t N, int64_t G) { return int(N * G < kRows ? (N * G + 1) / 2 * 2 : kRows); }

// Copies of the block's rows in a tile: those that fit a half or a quarter of it are there
// twice or four times.  2048 items of 1 to 2048 positions at D = 128, 16 rows: 126, 98, 86 us
// with one, two, four; 32 items of 48000 at D = 64, 56 rows: 85 us with one, 77 with two.
// (One token over 4096 positions, 2 tiles a CTA, would gain by one copy: 14.5 us for 15.3.)
int copies_for(int64_t N, int64_t G) { return N * G <= 32 ? 4 : N * G <= 64 ? 2 : 1; }

size_t workspace_for(int32_t N, int32_t G, int32_t D) {
    const size_t ctas = size_t(ctas_for(D, kMaxSms));
    return ctas * sizeof(Meta) +
           ctas * 2 * size_t(D + 2) * size_t(part_rows_for(N, G)) * sizeof(float);
}

using EncodeTiled = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                                 const cuuint64_t *, const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave,
                                 CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

int encode_fn(EncodeTiled *out) {
    static std::atomic<EncodeTiled> known{nullptr};
    EncodeTiled fn = known.load(std::memory_order_acquire);
    if (!fn) {
        void *f = nullptr;
        cudaDriverEntryPointQueryResult st;
        const cudaError_t e = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &st);
        if (e != cudaSuccess) return cuda_fail(e, "cuTensorMapEncodeTiled");
        if (st != cudaDriverEntryPointSuccess || !f) return cuda_fail(cudaErrorNotSupported, "cuTensorMapEncodeTiled");
        fn = reinterpret_cast<EncodeTiled>(f);
        known.store(fn, std::memory_order_release);
    }
    *out = fn;
    return LOOKUP_DRAFT_OK;
}

// The cache as rows of D elements; a box is 64 columns by one page's rows of a tile.
int cache_map(EncodeTiled fn, CUtensorMap *map, const void *base, int32_t type, int D, int64_t rows, int box_rows) {
    const cuuint64_t dims[2] = {cuuint64_t(D), cuuint64_t(rows)};
    const cuuint64_t strides[1] = {cuuint64_t(D) * 2};
    const cuuint32_t box[2] = {64, cuuint32_t(box_rows)}, elem[2] = {1, 1};
    const CUresult e =
        fn(map, type == LOOKUP_TYPE_F16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2,
           const_cast<void *>(base), dims, strides, box, elem, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
           CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return e == CUDA_SUCCESS ? LOOKUP_DRAFT_OK : cuda_fail(cudaErrorInvalidValue, "cuTensorMapEncodeTiled");
}

template <typename T, int D>
int launch(Params &p, cudaStream_t stream) {
    using S = Shape<D>;
    const int64_t items = int64_t(p.B) * p.Hkv * ((int64_t(p.N) * p.G + kRows - 1) / kRows);
    const int copies = copies_for(p.N, p.G);
    auto kernel = copies == 4 ? attention_kernel<T, D, 4> : copies == 2 ? attention_kernel<T, D, 2> : attention_kernel<T, D, 1>;
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, S::kSmem);
    if (e != cudaSuccess) return cuda_fail(e, "shared-memory opt-in");
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(p.ctas);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = S::kSmem;
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    cudaError_t r = cudaLaunchKernelEx(&cfg, kernel, p);
    if (r != cudaSuccess) return cuda_fail(r, "kernel launch");
    lookup_note_launch();
    // The join.  With about as many items as ranges each is cut once or twice, and a few
    // CTAs an item do (256 items of 128 rows: the whole call 506 us, and 514 with 16); a few
    // long items have tens of parts and take 16 (32 items of 56 rows at D = 64: 79 us, and 90
    // with 4).  A CTA takes four rows at a time; one where all items together have few rows
    // (8 items of 16 rows at D = 256: 19.1 us, and 20.4 by fours; 4 of 128 rows: 41 us by fours,
    // and 62).  Where those CTAs times the ranges would be several waves of mostly idle ones,
    // fewer CTAs share the ranges (those 32 items: 79 us, and 83 with CTAs for each range; an
    // odd number: evenly cut items begin at even distances).  1216: eight for each of 152 SMs.
    const bool single = items * p.part_rows < 512;
    const int per = std::min(single ? p.part_rows : (p.part_rows + 3) / 4, 3 * items >= p.ctas ? 4 : 16);
    const int64_t over = int64_t(per) * p.ctas <= 1216 ? p.ctas : std::min<int64_t>(p.ctas, 2 * items + 1);
    cfg.gridDim = dim3(unsigned(over), per);
    cfg.blockDim = dim3(kJoinThreads);
    cfg.dynamicSmemBytes = 0;
    r = cudaLaunchKernelEx(&cfg, single ? join_kernel<T, D, 1> : join_kernel<T, D, 4>, p);
    if (r != cudaSuccess) return cuda_fail(r, "kernel launch");
    lookup_note_launch();
    return LOOKUP_DRAFT_OK;
}

template <typename T>
int launch_d(Params &p, int D, cudaStream_t stream) {
    return D == 64 ? launch<T, 64>(p, stream) : D == 128 ? launch<T, 128>(p, stream) : launch<T, 256>(p, stream);
}

bool misaligned(const void *p, size_t to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) != 0; }

}  // namespace

extern "C" {

size_t lookup_paged_attention_workspace_bytes(int32_t B, int32_t N, int32_t Hq, int32_t Hkv, int32_t D) {
    if (B < 0 || N < 0 || Hq < 1 || Hkv < 1 || Hq % Hkv || (D != 64 && D != 128 && D != 256)) return 0;
    return workspace_for(N, Hq / Hkv, D);
}

int lookup_paged_attention(const void *q, const int64_t *q_strides, const void *k_cache, const void *v_cache,
                           const int32_t *block_table, const int32_t *kv_len, const int32_t *q_len, int32_t B,
                           int32_t N, int32_t Hq, int32_t Hkv, int32_t D, int32_t max_pages, int32_t pages,
                           int32_t page_size, float scale, int32_t window, int32_t type, void *out, float *lse,
                           void *workspace, size_t workspace_bytes, struct CUstream_st *stream) {
    lkd::TraceRange trace_("lookup_paged_attention");
    if (B < 0 || N < 0 || Hq < 1 || Hkv < 1 || Hq % Hkv || (D != 64 && D != 128 && D != 256) || max_pages < 1 ||
        pages < 1 || page_size < 8 || page_size > 1024 || (page_size & (page_size - 1)) || window < 0 ||
        !(std::fabs(scale) < INFINITY) || (type != LOOKUP_TYPE_F16 && type != LOOKUP_TYPE_BF16))
        return LOOKUP_DRAFT_EINVAL;
    const int64_t cache_rows = int64_t(pages) * Hkv * page_size;
    if (cache_rows > INT32_MAX - 128 || int64_t(max_pages) * page_size > INT32_MAX - 128)
        return LOOKUP_DRAFT_EINVAL;
    if (B == 0 || N == 0) return LOOKUP_DRAFT_OK;
    const int64_t rows = int64_t(B) * N * Hq;
    if (int64_t(N) * Hq > (1 << 30) || rows > (int64_t(1) << 30)) return LOOKUP_DRAFT_EINVAL;
    if (!q || !q_strides || !k_cache || !v_cache || !block_table || !kv_len || !out || !workspace)
        return LOOKUP_DRAFT_EINVAL;
    for (const void *x : {q, k_cache, v_cache, static_cast<const void *>(workspace), static_cast<const void *>(out)})
        if (misaligned(x, 16)) return LOOKUP_DRAFT_EINVAL;
    const int64_t axes[3] = {B, N, Hq};
    for (int k = 0; k < 3; ++k)                              // (an axis of one has any stride: it is not used)
        if (axes[k] > 1 && (q_strides[k] & 7)) return LOOKUP_DRAFT_EINVAL;
    if (misaligned(block_table, 4) || misaligned(kv_len, 4) || misaligned(q_len, 4) || misaligned(lse, 4))
        return LOOKUP_DRAFT_EINVAL;
    const int G = Hq / Hkv;
    if (workspace_bytes < workspace_for(N, G, D)) return LOOKUP_DRAFT_EINVAL;
    int sms = 0;
    int rc = lkd::sm_count(&sms);
    if (rc != LOOKUP_DRAFT_OK) return rc;
    Params p{};
    EncodeTiled fn = nullptr;
    rc = encode_fn(&fn);
    const int tile = D == 64 ? Shape<64>::kTile : D == 128 ? Shape<128>::kTile : Shape<256>::kTile;
    const int box_rows = page_size < tile ? page_size : tile;
    if (rc == LOOKUP_DRAFT_OK) rc = cache_map(fn, &p.k_map, k_cache, type, D, cache_rows, box_rows);
    if (rc == LOOKUP_DRAFT_OK) rc = cache_map(fn, &p.v_map, v_cache, type, D, cache_rows, box_rows);
    if (rc != LOOKUP_DRAFT_OK) return rc;
    p.q = q, p.qb = q_strides[0], p.qn = q_strides[1], p.qh = q_strides[2];
    p.table = block_table, p.kv_len = kv_len, p.q_len = q_len;
    p.B = B, p.N = N, p.Hq = Hq, p.Hkv = Hkv, p.G = G, p.max_pages = max_pages, p.pages = pages;
    while ((1 << p.page_shift) < page_size) ++p.page_shift;
    p.window = window, p.ctas = ctas_for(D, sms < kMaxSms ? sms : kMaxSms), p.part_rows = part_rows_for(N, G);
    p.cache_rows = int32_t(cache_rows);
    p.c = std::fabs(scale) * 1.4426950408889634f;
    p.negate = scale < 0.0f;
    p.out = out, p.lse = lse;
    p.meta = static_cast<Meta *>(workspace);
    p.parts = reinterpret_cast<float *>(p.meta + p.ctas);
    p.limit = 2 * lookup_wait_limit_ns();        // at 2 GHz

    return type == LOOKUP_TYPE_F16 ? launch_d<__half>(p, D, stream) : launch_d<__nv_bfloat16>(p, D, stream);
}

}  // extern "C"
