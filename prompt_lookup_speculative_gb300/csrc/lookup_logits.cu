// lookup_logits.cu -- verification of proposal blocks against the target's logits.
//
// The contract is in include/lookup_target.h (lookup_verify_logits).
//
// The mathematics: p(t) = exp((x_t - m) / T) / s with m the row's maximum and s the sum
// of the weights, in one pass with a running m: parts (m, s) of a row join as M = max m,
// sum s exp((m - M) / T).  A proposal d is accepted when u q(d) < p(d).  The token at the
// first rejection is drawn from the residual max(p - q, 0), the bonus token from p, by a
// race: the largest of (p - q)(t) / e_t over exponential noise e is at t with that
// probability, and needs no normalisation and no prefix sums over the vocabulary.
//
// What bounds it: the logits' bytes, each row of 0.3 to 0.6 MB read once.  Two kernels:
// stats_kernel streams every row that a proposal is tested in, cut into segments so
// that a few rows fill the device, and leaves per segment the running maximum m,
// s = sum exp((x - m) / T) and (greedy requests) the lowest index of m.
// pick_kernel, a cluster of CTAs per request, joins a request's segments, finds its
// first rejected position and reads that one row again, with the noise, for the race
// that draws its token.  The race needs p(t) - q(t) and so the whole row's sum
// before its first comparison; a second look at one row of P + 1 is cheaper than
// carrying every row's race through the first pass, where it would read the noise
// P + 1 times and double the instructions per logit.
//
// 64 blocks of 16 over 151936 bf16 logits: 56 us for 272 MB (4.9 TB/s, 72% of a copy's
// rate), 43 of them the streaming and 13 the draws, which wait for the first kernel's
// last row and then for a row and its noise.  64 blocks of 8 with a draft distribution
// over float32 logits 58 us (5.3 TB/s).  8 blocks of 16 over 32000 logits 11.3 us, 8.0 of
// them without the race; one block 8.8, and 5.9 without: there both kernels are latency.

#include "lookup_draft.h"
#include "lookup_target.h"
#include "common.cuh"

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cfloat>
#include <cmath>
#include <cstdint>
#include <type_traits>

namespace {

using lkd::allow_dependent_launch;
using lkd::kMaxBlock;
using lkd::launch_pdl;
using lkd::wait_for_prerequisite_grid;

constexpr int kStatWarps = 16;           // of a CTA of stats_kernel, each with a ring of its own
constexpr int kStatThreads = 32 * kStatWarps;
constexpr int kPer = 8;                  // 16-byte pieces of a lane and tile
constexpr int kTile = 32 * kPer;         // pieces of a tile: 4 KB, one bulk copy
constexpr int kRing = 3;                 // tiles in flight per warp: 192 KB per SM
constexpr int kSegTiles = 4;             // tiles of a segment at most (64 blocks of 16 over 151936: 56 us; 8: 58, 2: 61)
constexpr int kMaxCtas = 160;            // CTAs of stats_kernel at most, one per SM
constexpr float kFused = 2048.0f;        // |m c| up to which the weights take one fused operation each
constexpr int kPickThreads = 512;
constexpr int kKept = 32;                // positions whose statistics a CTA of pick_kernel keeps
constexpr int kMaxCluster = 8;           // CTAs per request in pick_kernel at most
constexpr int kRace = 16;                // logits in flight per thread there (8: those blocks 62 us)
constexpr int kMaxV = 1 << 30;

struct Params {
    const int32_t *block, *len;
    const void *logits;
    int64_t lb, lp;                      // strides of logits: request, position (elements)
    const float *noise, *temperature, *u, *qprobs;
    int64_t qb, qp;                      // strides of qprobs
    const int32_t *point_mass;
    int32_t B, P, V, segs, cluster;
    int32_t *out_accepted, *out_commit, *out_ncommit;
    float *out_logprobs;
    float4 *part;                        // [B][P + 1][segs]: m, s, index of m (bits), unused
    int32_t *status;                     // [ctas]: not 0 where a wait of stats_kernel ran out
    int32_t ctas;
    uint64_t limit;                      // clocks that a wait may take
};

__device__ inline float to_f32(float x) { return x; }
__device__ inline float to_f32(__half x) { return __half2float(x); }
__device__ inline float to_f32(__nv_bfloat16 x) { return __bfloat162float(x); }

// A logit as the contract reads it: NaN is -infinity.
template <typename T>
__device__ inline float logit(const T *row, int64_t i) {
    const float x = to_f32(row[i]);
    return x != x ? -INFINITY : x;
}

// Weight of logit x under the row's maximum m: 1 at the maximum (also where both
// are infinite), 0 at -infinity, exp((x - m) / T) between.
__device__ inline float weight(float x, float m, float inv_t) {
    if (x == m) return 1.0f;
    return x == -INFINITY ? 0.0f : expf((x - m) * inv_t);
}

// Greedy: no noise, or a temperature that is not a positive finite number.
__device__ inline bool is_greedy(const Params &p, int b) {
    if (!p.noise) return true;
    if (!p.temperature) return false;
    const float t = p.temperature[b];
    return !(t > 0.0f && t <= FLT_MAX);
}

__device__ inline float inv_temperature(const Params &p, int b) {
    return (is_greedy(p, b) || !p.temperature) ? 1.0f : 1.0f / p.temperature[b];
}

// A row part's maximum (empty: -infinity), the sum of its weights under that
// maximum, and the maximum's lowest index.
struct Stat {
    float m, s;
    int32_t at;
};

__device__ inline Stat join(const Stat &a, const Stat &b, float inv_t) {
    if (a.m == -INFINITY) return b;
    if (b.m == -INFINITY) return a;
    Stat r;
    r.m = fmaxf(a.m, b.m);
    r.s = a.s * weight(a.m, r.m, inv_t) + b.s * weight(b.m, r.m, inv_t);
    r.at = a.m == b.m ? min(a.at, b.at) : (a.m > b.m ? a.at : b.at);
    return r;
}

// The warp's lanes as one: the maximum first, one factor per lane, then the sum (and
// the index, where it is wanted); every lane gets the result.
__device__ inline Stat warp_join(Stat v, float inv_t, bool index) {
    float m = v.m;
#pragma unroll
    for (int d = 16; d; d >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
    float s = v.m == -INFINITY ? 0.0f : v.s * weight(v.m, m, inv_t);
#pragma unroll
    for (int d = 16; d; d >>= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
    const int32_t at = index ? __reduce_min_sync(0xffffffffu, v.m == m ? v.at : INT32_MAX) : INT32_MAX;
    return Stat{m, s, at};
}

// Word k of a piece of 16 bytes as two logits (float32: words 2k and 2k + 1).
__device__ inline float2 two(const uint4 &v, int k, float) {
    return k ? make_float2(__uint_as_float(v.z), __uint_as_float(v.w))
             : make_float2(__uint_as_float(v.x), __uint_as_float(v.y));
}
__device__ inline uint32_t word(const uint4 &v, int k) { return k == 0 ? v.x : k == 1 ? v.y : k == 2 ? v.z : v.w; }
__device__ inline float2 two(const uint4 &v, int k, __nv_bfloat16) {
    return make_float2(__uint_as_float(word(v, k) << 16), __uint_as_float(word(v, k) & 0xffff0000u));
}
__device__ inline float2 two(const uint4 &v, int k, __half) {
    const uint32_t w = word(v, k);
    return __half22float2(*reinterpret_cast<const __half2 *>(&w));
}

// The largest logit of two pieces, word by word (a NaN loses to any number).
__device__ inline uint4 max_words(const uint4 &a, const uint4 &b, float) {
    return make_uint4(__float_as_uint(fmaxf(__uint_as_float(a.x), __uint_as_float(b.x))),
                      __float_as_uint(fmaxf(__uint_as_float(a.y), __uint_as_float(b.y))),
                      __float_as_uint(fmaxf(__uint_as_float(a.z), __uint_as_float(b.z))),
                      __float_as_uint(fmaxf(__uint_as_float(a.w), __uint_as_float(b.w))));
}
__device__ inline uint32_t max_pair(uint32_t a, uint32_t b, __half) {
    uint32_t d;
    asm("max.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}
__device__ inline uint32_t max_pair(uint32_t a, uint32_t b, __nv_bfloat16) {
    uint32_t d;
    asm("max.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}
template <typename T>
__device__ inline uint4 max_words(const uint4 &a, const uint4 &b, T t) {
    return make_uint4(max_pair(a.x, b.x, t), max_pair(a.y, b.y, t), max_pair(a.z, b.z, t), max_pair(a.w, b.w, t));
}

__device__ inline float exp2_approx(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Two float32 operations in one instruction.
__device__ inline float2 add2(float2 a, float2 b) {
    float2 d;
    asm("{\n\t.reg .b64 x, y, z;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\t"
        "add.rn.f32x2 z, x, y;\n\tmov.b64 {%0, %1}, z;\n\t}"
        : "=f"(d.x), "=f"(d.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return d;
}
__device__ inline float2 fma2(float2 a, float2 b, float2 c) {
    float2 d;
    asm("{\n\t.reg .b64 x, y, z, w;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\tmov.b64 z, {%6, %7};\n\t"
        "fma.rn.f32x2 w, x, y, z;\n\tmov.b64 {%0, %1}, w;\n\t}"
        : "=f"(d.x), "=f"(d.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
    return d;
}
__device__ inline float2 mul2(float2 a, float2 b) {
    float2 d;
    asm("{\n\t.reg .b64 x, y, z;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\t"
        "mul.rn.f32x2 z, x, y;\n\tmov.b64 {%0, %1}, z;\n\t}"
        : "=f"(d.x), "=f"(d.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return d;
}

struct StatSmem {
    uint64_t full[kStatWarps][kRing];
    uint32_t next, failed;
};

// Every row that a proposal is tested in, once.  One CTA per SM; its warps take one of the
// CTA's segments after another (every ctas-th of all of them), each on its own: a warp
// streams its segment by bulk copies through a ring of three tiles, so that 192 KB per SM
// are in flight however far the warps have come, and nothing waits for a neighbour.
// (CTAs of 256 threads that load a segment into registers and then compute took 52 us
// for 233 MB of bf16 logits, and a ring shared by the CTA's warps 60 us: there each
// tile's chain of wait, maximum, weights and sum was on everyone's path.)  A row is taken
// in aligned pieces of 16 bytes; the first and the last may be part of the row only, and
// lanes add those logits by themselves.  Per tile the maximum first, in the type itself,
// then one factor for the sum so far, then the weights as 2^((x - m) c), c = log2(e) / T.
// While |m c| is at most 2^11 that is 2^(x c - m c), one fused operation: the product m c
// is rounded first, by err of at most 2^-14, which shifts all weights by one factor, and the
// sum is brought back by 1 - err ln 2 (right to 1e-9).  Past that (low temperatures, large
// logits) err can be any number, so the difference comes first, which rounds relative to
// itself: 64 blocks of 16 over 151936 take 57.1 us that way and 55.6 by the fused one.
template <typename T>
__global__ void __launch_bounds__(kStatThreads, 1) stats_kernel(const __grid_constant__ Params p) {
    constexpr int E = 16 / int(sizeof(T));               // logits of a piece
    extern __shared__ __align__(128) uint4 rings[];      // [kStatWarps][kRing][kTile]
    __shared__ StatSmem sm;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    volatile uint32_t *failed = &sm.failed;
    uint4 *ring = rings + warp * kRing * kTile;
    if (tid == 0) {
        sm.next = 0;
        sm.failed = 0;
    }
    if (lane == 0) {
        for (int k = 0; k < kRing; ++k) lkd::mbar_init(lkd::smem_addr(&sm.full[warp][k]), 1);
        lkd::fence_barrier_init();
    }
    __syncthreads();
    wait_for_prerequisite_grid();
    allow_dependent_launch();
    const uint32_t units = uint32_t(p.B) * uint32_t(p.P + 1) * uint32_t(p.segs);
    const uint32_t none = std::is_same<T, float>::value ? 0xff800000u
                          : std::is_same<T, __half>::value ? 0xfc00fc00u : 0xff80ff80u;
    int at = 0;                                          // the ring's next tile to use, and its parity
    uint32_t phase = 0;
    bool ok = true;
    while (ok) {
        uint32_t u = 0;
        if (lane == 0) u = atomicAdd(&sm.next, 1u);
        u = blockIdx.x + __shfl_sync(0xffffffffu, u, 0) * uint32_t(p.ctas);
        if (u >= units) break;
        const uint32_t row_id = u / uint32_t(p.segs);
        const int seg = int(u - row_id * uint32_t(p.segs));
        const int b = int(row_id / uint32_t(p.P + 1)), i = int(row_id - uint32_t(b) * uint32_t(p.P + 1));
        const int n = p.len[b];
        if (i > n || n > p.P) continue;                 // a row no proposal is tested in
        const T *row = static_cast<const T *>(p.logits) + b * p.lb + i * p.lp;
        const int mis = int((reinterpret_cast<uintptr_t>(row) & 15) / sizeof(T));    // logits before the row in piece 0
        const int pieces = (p.V + mis + E - 1) / E;
        const int per = int((uint32_t(pieces) + uint32_t(p.segs) - 1) / uint32_t(p.segs));
        const int lo = min(seg * per, pieces), hi = min(lo + per, pieces);
        // pieces [first, last) are all the row's: the ones that bulk copies bring
        const int first = max(lo, mis ? 1 : 0), last = max(min(hi, (p.V + mis) / E), first);
        const int tiles = (last - first + kTile - 1) / kTile;
        const uint4 *base = reinterpret_cast<const uint4 *>(row - mis) + first;
        auto fetch = [&](int t, int to) {                // by one lane: tile t into place `to`
            const uint32_t bytes = uint32_t(min(kTile, last - first - t * kTile)) * 16;
            const uint32_t bar = lkd::smem_addr(&sm.full[warp][to]);
            lkd::mbar_expect_tx(bar, bytes);
            lkd::bulk_copy_g2s_stream(lkd::smem_addr(ring + to * kTile), base + t * kTile, bytes, bar);
        };
        if (lane == 0)
            for (int t = 0; t < min(tiles, kRing); ++t) fetch(t, (at + t) % kRing);
        const bool greedy = is_greedy(p, b);
        const float inv_t = inv_temperature(p, b), c = inv_t * 1.4426950408889634f;
        Stat v{-INFINITY, 0.0f, INT32_MAX};
        // the row's first and last logits, short of a piece: a lane each, at most 2 (E - 1)
        {
            const int head = mis ? min(E - mis, p.V) : 0, tail = max((p.V + mis) / E * E - mis, head);
            const int j = lane < E ? lane : tail + lane - E;
            const bool mine = lane < E ? lo == 0 && lane < head : hi == pieces && lo < hi && lane < 2 * E && j < p.V;
            const float x = mine ? logit(row, j) : -INFINITY;
            if (x > -INFINITY) v = Stat{x, 1.0f, j};
        }
        for (int t = 0; ok && t < tiles; ++t) {
            ok = __all_sync(0xffffffffu, lkd::wait(lkd::smem_addr(&sm.full[warp][at]), phase, failed, p.limit));
            if (!ok) {                                   // no copy outlives the CTA
                for (int k = 0; k < min(tiles - t, kRing); ++k) {
                    const uint64_t until = lkd::global_ns() + 1000000000ull;
                    while (!lkd::mbar_try_wait(lkd::smem_addr(&sm.full[warp][at]), phase) && lkd::global_ns() < until) {
                    }
                    if (++at == kRing) {
                        at = 0;
                        phase ^= 1;
                    }
                }
                break;
            }
            const int count = min(kTile, last - first - t * kTile);
            uint4 r[kPer];
#pragma unroll
            for (int k = 0; k < kPer; ++k) r[k] = ring[at * kTile + k * 32 + lane];
            __syncwarp();
            if (lane == 0 && t + kRing < tiles) fetch(t + kRing, at);
            if (++at == kRing) {
                at = 0;
                phase ^= 1;
            }
            if (count < kTile) {                         // (past the copy the ring holds older logits)
#pragma unroll
                for (int k = 0; k < kPer; ++k)
                    if (k * 32 + lane >= count) r[k] = make_uint4(none, none, none, none);
            }
            uint4 top = r[0];
#pragma unroll
            for (int k = 1; k < kPer; ++k) top = max_words(top, r[k], T());
            float big = -INFINITY;
#pragma unroll
            for (int w = 0; w < E / 2; ++w) {
                const float2 x = two(top, w, T());
                big = fmaxf(big, fmaxf(x.x, x.y));
            }
            if (big > v.m) {
                v.s = v.m == -INFINITY ? 0.0f : v.s * weight(v.m, big, inv_t);
                v.m = big;
                v.at = INT32_MAX;
            }
            if (greedy && big == v.m) {                  // the lowest index so far of the lane's maximum
#pragma unroll
                for (int k = kPer - 1; k >= 0; --k)
#pragma unroll
                    for (int w = E / 2 - 1; w >= 0; --w) {
                        const float2 x = two(r[k], w, T());
                        const int j = (first + t * kTile + k * 32 + lane) * E + 2 * w - mis;
                        if (x.y == big) v.at = min(v.at, j + 1);
                        if (x.x == big) v.at = min(v.at, j);
                    }
            }
            const float mc = v.m * c;
            const float2 cc = make_float2(c, c);
            auto weights = [&](auto difference) {
                const float2 minus = decltype(difference)::value ? make_float2(-v.m, -v.m) : make_float2(-mc, -mc);
                float2 s0 = make_float2(0.0f, 0.0f), s1 = s0;
#pragma unroll
                for (int k = 0; k < kPer; ++k)
#pragma unroll
                    for (int w = 0; w < E / 2; ++w) {
                        const float2 x = two(r[k], w, T());
                        const float2 a = decltype(difference)::value ? mul2(add2(x, minus), cc) : fma2(x, cc, minus);
                        const float2 e = make_float2(exp2_approx(a.x), exp2_approx(a.y));
                        if (w & 1) s1 = add2(s1, e);
                        else s0 = add2(s0, e);
                    }
                return (s0.x + s0.y) + (s1.x + s1.y);
            };
            float sum;
            if (fabsf(mc) <= kFused) {
                // mc is m c rounded, off by err: every weight is 2^err too large, so the sum is
                const float err = fmaf(v.m, c, -mc);
                sum = weights(std::false_type());
                sum = fmaf(sum, err * -0.6931471805599453f, sum);
            } else {
                sum = weights(std::true_type());
            }
            if (!(sum <= FLT_MAX)) {                     // infinities or NaN among them: one by one
                sum = 0.0f;
#pragma unroll
                for (int k = 0; k < kPer; ++k)
#pragma unroll
                    for (int w = 0; w < E / 2; ++w) {
                        const float2 x = two(r[k], w, T());
                        if (x.x > -INFINITY) sum += weight(x.x, v.m, inv_t);
                        if (x.y > -INFINITY) sum += weight(x.y, v.m, inv_t);
                    }
            }
            v.s += sum;
        }
        const Stat all = warp_join(v, inv_t, greedy);
        if (lane == 0 && ok) p.part[u] = make_float4(all.m, all.s, __int_as_float(all.at), 0.0f);
    }
    __syncthreads();
    if (tid == 0) p.status[blockIdx.x] = int32_t(sm.failed);
}

// Row (b, i)'s statistics from its segments, by one warp (every lane gets them).
__device__ inline Stat row_stat(const Params &p, int b, int i, float inv_t, int lane) {
    const float4 *part = p.part + (int64_t(b) * (p.P + 1) + i) * p.segs;
    Stat v{-INFINITY, 0.0f, INT32_MAX};
#pragma unroll 4
    for (int k = lane; k < p.segs; k += 32) {
        const float4 q = part[k];
        v = join(v, Stat{q.x, q.y, __float_as_int(q.z)}, inv_t);
    }
    return warp_join(v, inv_t, true);
}

// The best race key so far: the largest, at its lowest index.
struct Best {
    float key;
    int32_t at;
};

__device__ inline Best better(const Best &a, const Best &b) {
    if (a.key != b.key) return a.key > b.key ? a : b;
    return a.at <= b.at ? a : b;
}

__device__ inline Best warp_better(Best v) {
#pragma unroll
    for (int d = 16; d; d >>= 1) {
        Best o;
        o.key = __shfl_xor_sync(0xffffffffu, v.key, d);
        o.at = __shfl_xor_sync(0xffffffffu, v.at, d);
        v = better(v, o);
    }
    return v;
}

__device__ inline uint32_t cluster_rank() {
    uint32_t r;
    asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ inline void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ inline void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }
// Writes 8 bytes to the same shared-memory place of the cluster's CTA `rank`.
__device__ inline void store_to(uint32_t rank, void *place, uint64_t v) {
    uint32_t at;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(lkd::smem_addr(place)), "r"(rank));
    asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(at), "l"(v) : "memory");
}

// The best of the whole cluster, in every thread of it.  `place` is written by every
// CTA of the cluster and used once per launch.
__device__ inline Best cluster_best(Best v, uint64_t (&warps)[kPickThreads / 32], uint64_t (&place)[kMaxCluster],
                                    int rank, int cluster) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    auto pack = [](const Best &b) { return (uint64_t(__float_as_uint(b.key)) << 32) | uint32_t(b.at); };
    auto unpack = [](uint64_t w) { return Best{__uint_as_float(uint32_t(w >> 32)), int32_t(uint32_t(w))}; };
    v = warp_better(v);
    if (lane == 0) warps[warp] = pack(v);
    __syncthreads();
    if (warp == 0) {
        v = warp_better(lane < kPickThreads / 32 ? unpack(warps[lane]) : Best{0.0f, INT32_MAX});
        if (lane < cluster) store_to(lane, &place[rank], pack(v));
        __syncwarp();
    }
    cluster_arrive();
    cluster_wait();
    return warp_better(lane < cluster ? unpack(place[lane]) : Best{0.0f, INT32_MAX});
}

// One cluster per request.  Every CTA of it finds the first rejected position a (a
// warp per position: its segments joined, its proposal tested), then takes an equal
// part of row a's race, logit by logit across the threads (noise, q and the row have
// alignments of their own); CTA 0 takes the best and writes the outputs.
template <typename T>
__global__ void __launch_bounds__(kPickThreads) pick_kernel(const __grid_constant__ Params p) {
    __shared__ int s_first;
    __shared__ Stat kept[kKept], s_row;
    __shared__ uint64_t warps[3][kPickThreads / 32], places[3][kMaxCluster];
    const int b = blockIdx.x / p.cluster, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int rank = int(cluster_rank());
    const int per = int((uint32_t(p.V) + uint32_t(p.cluster) - 1) / uint32_t(p.cluster));
    const int lo = min(rank * per, p.V), hi = min(lo + per, p.V);    // this CTA's part of the race
    // the noise on its way while stats_kernel's last CTAs run: it is the call's input, and
    // this grid starts after all of stats_kernel's CTAs have waited for what came before
    if (p.noise)
        for (int j = lo + 32 * tid; j < hi; j += 32 * kPickThreads) lkd::prefetch_l2(p.noise + int64_t(b) * p.V + j);
    wait_for_prerequisite_grid();
    allow_dependent_launch();
    const int P = p.P, n = p.len[b];
    int32_t *commit = p.out_commit + int64_t(b) * (P + 1);
    float *lps = p.out_logprobs ? p.out_logprobs + int64_t(b) * (P + 1) : nullptr;
    // no valid block, or logits that did not arrive in time: an error row
    bool bad = tid < p.ctas && p.status[tid] != 0;
    static_assert(kMaxCtas <= kPickThreads, "a thread per CTA of stats_kernel");
    if (__syncthreads_or(bad || n < 0 || n > P)) {
        if (rank) return;
        for (int i = tid; i <= P; i += kPickThreads) {
            commit[i] = -1;
            if (lps) lps[i] = 0.0f;
        }
        if (tid == 0) {
            p.out_accepted[b] = -1;
            p.out_ncommit[b] = 0;
        }
        return;
    }
    const bool greedy = is_greedy(p, b);
    if (greedy && rank) return;                          // no race: CTA 0 does it all
    const float inv_t = inv_temperature(p, b);
    const T *rows = static_cast<const T *>(p.logits) + b * p.lb;
    const int32_t *block = p.block + int64_t(b) * P;
    if (tid == 0) s_first = n;
    __syncthreads();
    // a warp per position: is its proposal accepted, and with which probability
    for (int i = warp; i <= n; i += kPickThreads / 32) {
        const int d = i < n ? block[i] : -1;
        const float u = i < n && !greedy ? p.u[int64_t(b) * P + i] : 1.0f;
        const bool point = !p.qprobs || (i < n && p.point_mass && p.point_mass[int64_t(b) * P + i] != 0);
        const bool in = d >= 0 && d < p.V;
        const float x = in ? logit(rows + i * p.lp, d) : -INFINITY;
        const float q = point || !in ? 1.0f : p.qprobs[b * p.qb + i * p.qp + d];
        const Stat v = row_stat(p, b, i, inv_t, lane);
        if (lane == 0 && i < kKept) kept[i] = v;
        if (i == n) break;                               // past the block: nothing to test
        const bool fits = in && v.m > -INFINITY;
        const bool ok = greedy ? fits && d == v.at : __fmul_rn(u, q) < (fits ? weight(x, v.m, inv_t) / v.s : 0.0f);
        if (lane == 0) {
            if (!ok) atomicMin(&s_first, i);
            if (lps && !rank) lps[i] = ok ? (x == v.m ? 0.0f : (x - v.m) * inv_t) - logf(v.s) : 0.0f;
        }
    }
    __syncthreads();
    const int a = s_first;
    if (a < kKept) {
        if (tid == 0) s_row = kept[a];
    } else if (warp == 0) {
        const Stat v = row_stat(p, b, a, inv_t, lane);
        if (lane == 0) s_row = v;
    }
    __syncthreads();
    const Stat row = s_row;
    const T *x = rows + a * p.lp;
    int32_t token = row.m > -INFINITY ? row.at : -1;
    if (!greedy) {
        cluster_arrive();                                // every CTA runs before another writes to it
        const bool rejected = a < n;
        const bool point = !p.qprobs || (rejected && p.point_mass && p.point_mass[int64_t(b) * P + a] != 0);
        const int32_t d = rejected && point ? block[a] : -1;
        const float *q = rejected && !point ? p.qprobs + b * p.qb + a * p.qp : nullptr;
        const float *noise = p.noise + int64_t(b) * p.V;
        const float c = inv_t * 1.4426950408889634f, inv_s = 1.0f / row.s;
        Best best{0.0f, INT32_MAX};
        // keys without the common factor 1 / s where no q is taken off.  The best of
        // kRace keys first; which one it was only where it beats the thread's best.
        auto race = [&](auto kind) {
            constexpr bool with_q = decltype(kind)::value;
            for (int j0 = lo + tid; j0 < hi; j0 += kRace * kPickThreads) {
                float key[kRace], es[kRace], qs[kRace];
#pragma unroll
                for (int k = 0; k < kRace; ++k) {
                    const int j = min(j0 + k * kPickThreads, hi - 1);        // past the end: the last one again
                    key[k] = to_f32(x[j]);
                    es[k] = __ldcs(noise + j);
                    if (with_q) qs[k] = __ldcs(q + j);
                }
                float top = 0.0f;                        // NaN drops out
#pragma unroll
                for (int k = 0; k < kRace; ++k) {
                    const float w = exp2_approx((key[k] - row.m) * c);
                    key[k] = __fdividef(with_q ? fmaf(w, inv_s, -qs[k]) : w, es[k]);
                    top = fmaxf(top, key[k]);
                }
                if (top > best.key) {
#pragma unroll
                    for (int k = 0; k < kRace; ++k) {
                        const int j = min(j0 + k * kPickThreads, hi - 1);
                        if (key[k] > best.key && j != d) best = Best{key[k], j};
                    }
                }
            }
        };
        const bool plain = row.m > -INFINITY && row.m <= FLT_MAX && c <= FLT_MAX;
        if (plain) {
            if (q) race(std::true_type());
            else race(std::false_type());
        }
        __syncwarp();                                    // the cluster's barrier wants whole warps
        cluster_wait();
        best = cluster_best(best, warps[0], places[0], rank, p.cluster);
        if (best.key == 0.0f && row.m > -INFINITY) {
            // nothing left above 2^-126, or infinite logits: once more, to the smallest
            // float32, with p's own best should the residual be nothing at all
            Best all{0.0f, INT32_MAX};
            for (int j = lo + tid; j < hi; j += kPickThreads) {
                const float w = weight(logit(x, j), row.m, inv_t), own = w / noise[j];
                const float key = q ? (w / row.s - q[j]) / noise[j] : own;
                if (key > best.key && j != d) best = Best{key, j};
                if (own > all.key) all = Best{own, j};
            }
            best = cluster_best(best, warps[1], places[1], rank, p.cluster);
            all = cluster_best(all, warps[2], places[2], rank, p.cluster);
            if (best.key == 0.0f) best = all;
        }
        if (rank) return;
        token = best.key > 0.0f ? best.at : -1;
    }
    if (warp == 0) {
        for (int i = lane; i <= P; i += 32) {
            commit[i] = i < a ? block[i] : (i == a ? token : -1);
            if (lps && i >= a) {
                float v = 0.0f;
                if (i == a && token >= 0) {
                    const float z = logit(x, token);
                    v = (z == row.m ? 0.0f : (z - row.m) * inv_t) - logf(row.s);
                }
                lps[i] = v;
            }
        }
        if (lane == 0) {
            p.out_accepted[b] = a;
            p.out_ncommit[b] = a + (token >= 0);
        }
    }
}

// Segments of a row of `size`-byte logits: a tile each while there are fewer tiles than
// warps (on a GB300's 152 SMs), kSegTiles tiles at most.
int64_t segments(int32_t B, int32_t P, int32_t V, int size) {
    const int64_t tiles = (int64_t(V) * size / 16 + 2 + kTile - 1) / kTile;          // of a row
    const int64_t each = std::min<int64_t>(std::max<int64_t>(tiles * B * (P + 1) / (152 * kStatWarps), 1), kSegTiles);
    return (tiles + each - 1) / each;
}

// CTAs of a request's cluster: a power of two, one per 4096 logits of its race as
// long as all clusters run at once (304: two CTAs per SM).  64 requests with 4 CTAs each take
// 56 us in all, with 1 83 us, with 8 62; 8 requests over 32000 logits 11.5 us with 8, 17 with 1.
int cluster_for(int32_t B, int32_t V) {
    int c = 1;
    while (c < kMaxCluster && int64_t(c) * 4096 < V && int64_t(2) * c * B <= 304) c *= 2;
    return c;
}

template <typename T>
int launch(const Params &p, cudaStream_t stream) {
    constexpr size_t kBytes = size_t(kStatWarps) * kRing * kTile * 16;
    const cudaError_t opt = cudaFuncSetAttribute(stats_kernel<T>, cudaFuncAttributeMaxDynamicSharedMemorySize, int(kBytes));
    if (opt != cudaSuccess) return lookup_record_cuda_error(opt, "shared-memory opt-in");
    int rc = launch_pdl(stats_kernel<T>, unsigned(p.ctas), unsigned(kStatThreads), stream, p, kBytes);
    if (rc != LOOKUP_DRAFT_OK) return rc;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = unsigned(p.cluster);
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(unsigned(p.B) * unsigned(p.cluster));
    cfg.blockDim = dim3(kPickThreads);
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, pick_kernel<T>, p);
    if (e != cudaSuccess) return lookup_record_cuda_error(e, "kernel launch");
    lookup_note_launch();
    return LOOKUP_DRAFT_OK;
}

bool misaligned(const void *p, size_t to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) != 0; }

}  // namespace

extern "C" {

size_t lookup_verify_logits_workspace_bytes(int32_t B, int32_t P, int32_t V) {
    if (B < 0 || P < 0 || P > kMaxBlock || V < 1 || V >= kMaxV) return 0;
    return size_t(B) * size_t(P + 1) * size_t(std::max(segments(B, P, V, 4), segments(B, P, V, 2))) * sizeof(float4) +
           kMaxCtas * sizeof(int32_t);
}

int lookup_verify_logits(const int32_t *block, const int32_t *len, const void *logits, const int64_t *logits_strides,
                         int32_t type, int32_t V, const float *noise, const float *temperature, const float *u,
                         const float *qprobs, const int64_t *qprobs_strides, const int32_t *point_mass, int32_t B,
                         int32_t P, int32_t *out_accepted, int32_t *out_commit, int32_t *out_ncommit,
                         float *out_logprobs, void *workspace, size_t workspace_bytes, struct CUstream_st *stream) {
    lkd::TraceRange trace_("lookup_verify_logits");
    if (B < 0 || P < 0 || P > kMaxBlock || V < 1 || V >= kMaxV) return LOOKUP_DRAFT_EINVAL;
    if (type != LOOKUP_TYPE_F32 && type != LOOKUP_TYPE_F16 && type != LOOKUP_TYPE_BF16) return LOOKUP_DRAFT_EINVAL;
    if (B == 0) return LOOKUP_DRAFT_OK;
    const int64_t segs = segments(B, P, V, type == LOOKUP_TYPE_F32 ? 4 : 2);
    if (segs > INT32_MAX / (int64_t(B) * (P + 1)) || int64_t(B) * kMaxCluster > INT32_MAX) return LOOKUP_DRAFT_EINVAL;
    if ((P > 0 && !block) || !len || !logits || !logits_strides || !out_accepted || !out_commit || !out_ncommit ||
        !workspace)
        return LOOKUP_DRAFT_EINVAL;
    if (noise && P > 0 && (!u || (qprobs && !qprobs_strides))) return LOOKUP_DRAFT_EINVAL;
    if (misaligned(logits, type == LOOKUP_TYPE_F32 ? 4 : 2) || misaligned(workspace, 16)) return LOOKUP_DRAFT_EINVAL;
    for (const void *q : {static_cast<const void *>(block), static_cast<const void *>(len),
                          static_cast<const void *>(noise), static_cast<const void *>(temperature),
                          static_cast<const void *>(u), static_cast<const void *>(qprobs),
                          static_cast<const void *>(point_mass), static_cast<const void *>(out_accepted),
                          static_cast<const void *>(out_commit), static_cast<const void *>(out_ncommit),
                          static_cast<const void *>(out_logprobs)})
        if (misaligned(q, 4)) return LOOKUP_DRAFT_EINVAL;
    if (workspace_bytes < lookup_verify_logits_workspace_bytes(B, P, V)) return LOOKUP_DRAFT_EINVAL;
    const bool with_q = noise && qprobs && P > 0;
    int sms = 0;
    const int rc = lkd::sm_count(&sms);
    if (rc != LOOKUP_DRAFT_OK) return rc;
    Params p{};
    p.block = block, p.len = len, p.logits = logits, p.lb = logits_strides[0], p.lp = logits_strides[1];
    p.noise = noise, p.temperature = noise ? temperature : nullptr, p.u = u, p.qprobs = with_q ? qprobs : nullptr;
    if (with_q) p.qb = qprobs_strides[0], p.qp = qprobs_strides[1];
    p.point_mass = point_mass, p.B = B, p.P = P, p.V = V, p.segs = int32_t(segs), p.cluster = cluster_for(B, V);
    p.out_accepted = out_accepted, p.out_commit = out_commit, p.out_ncommit = out_ncommit, p.out_logprobs = out_logprobs;
    const int64_t units = int64_t(B) * (P + 1) * segs;
    p.ctas = int32_t(std::min<int64_t>(units, std::min(sms, kMaxCtas)));
    p.part = static_cast<float4 *>(workspace);
    p.status = reinterpret_cast<int32_t *>(p.part + units);
    p.limit = 2 * lookup_wait_limit_ns();                // at 2 GHz
    if (type == LOOKUP_TYPE_F32) return launch<float>(p, stream);
    if (type == LOOKUP_TYPE_F16) return launch<__half>(p, stream);
    return launch<__nv_bfloat16>(p, stream);
}

}  // extern "C"
