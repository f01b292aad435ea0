// lookup_kv_append.cu -- rotary positions and the append to the paged cache.
//
// The contract is in include/lookup_target.h (lookup_kv_append).
//
// The mathematics: a pair (a, b) of an element and its partner becomes (a cos t - b sin t,
// b cos t + a sin t), both products and the difference in float32, rounded once to the
// tensors' type.  The angles' cos and sin come from a table that the caller forms in 64
// bits, so any scaling of the frequencies is in it and no angle is computed here.
//
// What bounds it: the bytes of q, k and v, read once and written once.  One launch: each
// thread takes one unit of 16 elements of a head (for a rotated unit, the 8 pairs that
// share 8 angles) for kHeads heads of one token, so the angles are read once for them and
// all their 16-byte loads are in flight together.  The last CTAs report the requests with
// tokens that have no slot.  4 prompts of 8191 tokens, 32 query and 8 key-value heads of
// 128: 138 us (5.6 TB/s, 83% of a copy's rate); 64 blocks of 16 tokens 5.0 us, one token
// 2.3 us, which is the launch.  4096 blocks of 8 with 16 and 2 heads of 64 37 us (4.4 TB/s),
// whatever the layout of the pairs, the rotated part and the head's size; as four prompts
// 34 us: 7 us of start and end, then 5.9 TB/s, and the blocks' short runs of tokens.
//
// A head or a rotated part that is no multiple of 16 elements, and strides or addresses that
// are no multiples of 16 bytes, take a kernel of one pair of elements per thread: right for
// every case, and five to six times slower (796 us for those prompts, 183 for the blocks).

#include "lookup_draft.h"
#include "lookup_target.h"
#include "common.cuh"

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>

namespace {

using lkd::allow_dependent_launch;
using lkd::launch_pdl;
using lkd::wait_for_prerequisite_grid;

constexpr int kThreads = 256;
constexpr int kHeads = 2;                // heads of a thread (4 take more registers, and fewer threads fit: 158 us for 138)
constexpr int kMaxD = 1024;

struct Strides {
    int64_t b, n, h;
};

struct Params {
    const void *q, *k, *v;
    Strides qs, ks, vs;
    const int32_t *kv_len, *q_len, *table;
    const float *rotary;
    void *k_cache, *v_cache, *out_q;
    int32_t *status;
    int32_t B, N, Hq, Hkv, D, max_pages, pages, page_shift, rot, max_pos, interleaved;
    int32_t tokens;                      // of a CTA of append_units_kernel
    int32_t grid;                        // CTAs that append; the ones after them report
};

__device__ inline float to_f32(__half x) { return __half2float(x); }
__device__ inline float to_f32(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ inline void from_f32(float x, __half &y) { y = __float2half_rn(x); }
__device__ inline void from_f32(float x, __nv_bfloat16 &y) { y = __float2bfloat16_rn(x); }

__device__ inline int32_t clamped(int32_t x, int32_t lo, int32_t hi) { return min(max(x, lo), hi); }

__device__ inline int32_t block_tokens(const Params &p, int b) {
    return p.q_len ? clamped(p.q_len[b], 0, p.N) : p.N;
}

// The first row of the token's page for kv head 0 of the cache, plus its row in the
// page (add head * page_size for another head), or -1 where the token has no slot.
__device__ inline int64_t slot_of(const Params &p, int b, int64_t pos) {
    const int64_t at = pos >> p.page_shift;
    if (at >= p.max_pages || (p.rotary && pos >= p.max_pos)) return -1;
    const int32_t page = p.table[int64_t(b) * p.max_pages + at];
    if (page < 0 || page >= p.pages) return -1;
    return ((int64_t(page) * p.Hkv) << p.page_shift) + (pos & ((int64_t(1) << p.page_shift) - 1));
}

// status, by the CTAs after the appending ones: a warp per request, which looks at
// each page that the block's tokens touch.
__device__ inline void report(const Params &p) {
    const int lane = threadIdx.x & 31;
    const int64_t b = int64_t(blockIdx.x - p.grid) * (kThreads / 32) + (threadIdx.x >> 5);
    if (b >= p.B) return;
    const int n = block_tokens(p, int(b));
    const int64_t first = max(p.kv_len[b], 0), end = first + n;
    bool bad = n > 0 && p.rotary && end > p.max_pos;
    if (n > 0)
        for (int64_t at = (first >> p.page_shift) + lane; at <= ((end - 1) >> p.page_shift); at += 32) {
            const int32_t page = at < p.max_pages ? p.table[b * p.max_pages + at] : -1;
            bad |= page < 0 || page >= p.pages;
        }
    bad = __any_sync(0xffffffffu, bad);
    if (lane == 0) p.status[b] = bad ? 1 : 0;
}

__device__ inline float2 unpack2(uint32_t w, __half) { return __half22float2(*reinterpret_cast<const __half2 *>(&w)); }
__device__ inline float2 unpack2(uint32_t w, __nv_bfloat16) {
    return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}
__device__ inline uint32_t pack2(float lo, float hi, __half) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&h);
}
__device__ inline uint32_t pack2(float lo, float hi, __nv_bfloat16) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&h);
}

// Two words of a pair's unit rotated.  Half layout: x holds two a, y the two b that
// pair with them.  Interleaved: x and y each hold one pair.
template <typename T, bool INTER>
__device__ inline void turn(uint32_t &x, uint32_t &y, float c0, float s0, float c1, float s1) {
    const float2 f = unpack2(x, T()), g = unpack2(y, T());
    if (INTER) {
        x = pack2(f.x * c0 - f.y * s0, f.y * c0 + f.x * s0, T());
        y = pack2(g.x * c1 - g.y * s1, g.y * c1 + g.x * s1, T());
    } else {
        x = pack2(f.x * c0 - g.x * s0, f.y * c1 - g.y * s1, T());
        y = pack2(g.x * c0 + f.x * s0, g.y * c1 + f.y * s1, T());
    }
}

template <typename T, bool INTER>
__global__ void __launch_bounds__(kThreads, 4) append_units_kernel(const __grid_constant__ Params p) {
    wait_for_prerequisite_grid();
    allow_dependent_launch();
    if (int(blockIdx.x) >= p.grid) return report(p);
    const uint32_t units = p.D / 16;
    const int q_groups = p.q ? (p.Hq + kHeads - 1) / kHeads : 0, k_groups = p.k ? (p.Hkv + kHeads - 1) / kHeads : 0;
    const uint32_t per = units * (q_groups + 2 * k_groups);          // threads of a token
    const uint32_t tok0 = blockIdx.x * uint32_t(p.tokens);
    const int b0 = int(tok0 / uint32_t(p.N)), i0 = int(tok0 - uint32_t(b0) * uint32_t(p.N));
    for (uint32_t x = threadIdx.x; x < p.tokens * per; x += kThreads) {
        const uint32_t t = x / per, rest = x - t * per;
        int g = int(rest / units);
        const int u = int(rest - g * units);             // neighbouring threads: neighbouring units of a head
        int b = b0, i = i0 + int(t);
        for (; i >= p.N; i -= p.N) ++b;
        if (b >= p.B) return;
        const bool is_q = g < q_groups, is_k = !is_q && g < q_groups + k_groups;
        if (!is_q) g -= is_k ? q_groups : q_groups + k_groups;
        const int h0 = g * kHeads, heads = min(kHeads, (is_q ? p.Hq : p.Hkv) - h0);
        const int64_t pos = int64_t(max(p.kv_len[b], 0)) + i;
        const bool turned = u < p.rot / 16 && (is_q || is_k);
        // the unit's two 16-byte parts in a head
        int e0 = 16 * u, e1 = 16 * u + 8;
        if (!INTER && u < p.rot / 16) {
            e0 = 8 * u;
            e1 = p.rot / 2 + 8 * u;
        }
        // the loads first: they wait for nothing (rows past q_len are there, if unused)
        uint4 v0[kHeads], v1[kHeads];
        const Strides &st = is_q ? p.qs : is_k ? p.ks : p.vs;
        const T *src = static_cast<const T *>(is_q ? p.q : is_k ? p.k : p.v) + b * st.b + i * st.n + h0 * st.h;
#pragma unroll
        for (int k = 0; k < kHeads; ++k)
            if (k < heads) {
                v0[k] = __ldcs(reinterpret_cast<const uint4 *>(src + k * st.h + e0));
                v1[k] = __ldcs(reinterpret_cast<const uint4 *>(src + k * st.h + e1));
            }
        const int64_t slot = i < block_tokens(p, b) ? slot_of(p, b, pos) : -1;
        T *dst;
        int64_t step;
        if (is_q) {
            dst = static_cast<T *>(p.out_q) + ((int64_t(b) * p.N + i) * p.Hq + h0) * p.D;
            step = p.D;
        } else {
            if (slot < 0) continue;
            dst = static_cast<T *>(is_k ? p.k_cache : p.v_cache) + (slot + (int64_t(h0) << p.page_shift)) * p.D;
            step = int64_t(p.D) << p.page_shift;
        }
        if (slot < 0) {                                  // a query row past the block, or without a slot
#pragma unroll
            for (int k = 0; k < kHeads; ++k) v0[k] = v1[k] = make_uint4(0, 0, 0, 0);
        } else if (turned) {
            const float *row = p.rotary + pos * p.rot + 8 * u;
            const float4 c0 = *reinterpret_cast<const float4 *>(row), c1 = *reinterpret_cast<const float4 *>(row + 4);
            const float4 s0 = *reinterpret_cast<const float4 *>(row + p.rot / 2);
            const float4 s1 = *reinterpret_cast<const float4 *>(row + p.rot / 2 + 4);
#pragma unroll
            for (int k = 0; k < kHeads; ++k)
                if (k < heads) {
                    if (INTER) {                         // words of pairs 0 .. 3, then 4 .. 7
                        turn<T, INTER>(v0[k].x, v0[k].y, c0.x, s0.x, c0.y, s0.y);
                        turn<T, INTER>(v0[k].z, v0[k].w, c0.z, s0.z, c0.w, s0.w);
                        turn<T, INTER>(v1[k].x, v1[k].y, c1.x, s1.x, c1.y, s1.y);
                        turn<T, INTER>(v1[k].z, v1[k].w, c1.z, s1.z, c1.w, s1.w);
                    } else {                             // words of a and of b, two pairs each
                        turn<T, INTER>(v0[k].x, v1[k].x, c0.x, s0.x, c0.y, s0.y);
                        turn<T, INTER>(v0[k].y, v1[k].y, c0.z, s0.z, c0.w, s0.w);
                        turn<T, INTER>(v0[k].z, v1[k].z, c1.x, s1.x, c1.y, s1.y);
                        turn<T, INTER>(v0[k].w, v1[k].w, c1.z, s1.z, c1.w, s1.w);
                    }
                }
        }
#pragma unroll
        for (int k = 0; k < kHeads; ++k)
            if (k < heads) {
                *reinterpret_cast<uint4 *>(dst + k * step + e0) = v0[k];
                *reinterpret_cast<uint4 *>(dst + k * step + e1) = v1[k];
            }
    }
}

// One pair of elements of one head per thread.
template <typename T>
__global__ void __launch_bounds__(kThreads) append_pairs_kernel(const __grid_constant__ Params p) {
    wait_for_prerequisite_grid();
    allow_dependent_launch();
    if (int(blockIdx.x) >= p.grid) return report(p);
    const int half_d = (p.D + 1) / 2;
    const int heads = (p.q ? p.Hq : 0) + (p.k ? 2 * p.Hkv : 0);
    const int64_t idx = int64_t(blockIdx.x) * kThreads + threadIdx.x;
    const int64_t head_id = idx / half_d;
    const int e = int(idx - head_id * half_d);           // which pair of elements
    const int64_t tok = head_id / heads;
    int h = int(head_id - tok * heads);
    const int b = int(tok / p.N), i = int(tok - int64_t(b) * p.N);
    if (b >= p.B) return;
    const bool is_q = p.q && h < p.Hq;
    const int64_t pos = int64_t(max(p.kv_len[b], 0)) + i;
    const int64_t slot = i < block_tokens(p, b) ? slot_of(p, b, pos) : -1;
    if (!is_q && slot < 0) return;
    const T *src;
    T *dst;
    bool rotate = p.rotary != nullptr;
    if (is_q) {
        src = static_cast<const T *>(p.q) + b * p.qs.b + i * p.qs.n + h * p.qs.h;
        dst = static_cast<T *>(p.out_q) + (tok * p.Hq + h) * p.D;
    } else {
        if (p.q) h -= p.Hq;
        const bool is_k = h < p.Hkv;
        if (!is_k) h -= p.Hkv;
        const Strides &st = is_k ? p.ks : p.vs;
        src = static_cast<const T *>(is_k ? p.k : p.v) + b * st.b + i * st.n + h * st.h;
        dst = static_cast<T *>(is_k ? p.k_cache : p.v_cache) + (slot + (int64_t(h) << p.page_shift)) * p.D;
        rotate = rotate && is_k;
    }
    const int half = p.rot / 2;
    int j0 = 2 * e, j1 = 2 * e + 1;                      // the pair's elements
    if (rotate && e < half && !p.interleaved) {
        j0 = e;
        j1 = e + half;
    }
    T zero;
    from_f32(0.0f, zero);
    if (slot < 0) {                                      // a query row past the block, or without a slot
        dst[j0] = zero;
        if (j1 < p.D) dst[j1] = zero;
    } else if (rotate && e < half) {
        const float *row = p.rotary + pos * p.rot;
        const float c = row[e], s = row[half + e], x = to_f32(src[j0]), y = to_f32(src[j1]);
        from_f32(x * c - y * s, dst[j0]);
        from_f32(y * c + x * s, dst[j1]);
    } else {
        dst[j0] = src[j0];
        if (j1 < p.D) dst[j1] = src[j1];
    }
}

bool misaligned(const void *p, size_t to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) != 0; }

}  // namespace

extern "C" {

int lookup_kv_append(const void *q, const int64_t *q_strides, const void *k, const int64_t *k_strides, const void *v,
                     const int64_t *v_strides, const int32_t *kv_len, const int32_t *q_len,
                     const int32_t *block_table, int32_t B, int32_t N, int32_t Hq, int32_t Hkv, int32_t D,
                     int32_t max_pages, int32_t pages, int32_t page_size, const float *rotary, int32_t rot,
                     int32_t max_pos, int32_t interleaved, int32_t type, void *k_cache, void *v_cache, void *out_q,
                     int32_t *status, struct CUstream_st *stream) {
    lkd::TraceRange trace_("lookup_kv_append");
    if (B < 0 || N < 0 || Hq < 0 || Hkv < 1 || D < 1 || D > kMaxD || max_pages < 1 || pages < 1 || page_size < 1 ||
        (page_size & (page_size - 1)) || (q && Hq < 1))
        return LOOKUP_DRAFT_EINVAL;
    if (rotary && (rot < 2 || rot > D || (rot & 1) || max_pos < 1)) return LOOKUP_DRAFT_EINVAL;
    if (type != LOOKUP_TYPE_F16 && type != LOOKUP_TYPE_BF16) return LOOKUP_DRAFT_EINVAL;
    if (B == 0 || N == 0) return LOOKUP_DRAFT_OK;
    if (int64_t(B) * N > INT32_MAX) return LOOKUP_DRAFT_EINVAL;
    if (!kv_len || !block_table || !k != !v || (k && (!k_cache || !v_cache || !k_strides || !v_strides)) ||
        (q && (!out_q || !q_strides)))
        return LOOKUP_DRAFT_EINVAL;
    for (const void *x : {q, k, v, static_cast<const void *>(k_cache), static_cast<const void *>(v_cache),
                          static_cast<const void *>(out_q)})
        if (misaligned(x, 2)) return LOOKUP_DRAFT_EINVAL;
    for (const void *x : {static_cast<const void *>(kv_len), static_cast<const void *>(q_len),
                          static_cast<const void *>(block_table), static_cast<const void *>(rotary),
                          static_cast<const void *>(status)})
        if (misaligned(x, 4)) return LOOKUP_DRAFT_EINVAL;
    Params p{};
    p.q = q, p.k = k, p.v = v;
    auto strides = [&](const int64_t *s, int32_t heads) {    // an axis of one has any: it is not used
        return Strides{B > 1 ? s[0] : 0, N > 1 ? s[1] : 0, heads > 1 ? s[2] : 0};
    };
    if (q) p.qs = strides(q_strides, Hq);
    if (k) p.ks = strides(k_strides, Hkv);
    if (v) p.vs = strides(v_strides, Hkv);
    p.kv_len = kv_len, p.q_len = q_len, p.table = block_table, p.rotary = rotary;
    p.k_cache = k_cache, p.v_cache = v_cache, p.out_q = out_q, p.status = status;
    p.B = B, p.N = N, p.Hq = Hq, p.Hkv = Hkv, p.D = D, p.max_pages = max_pages, p.pages = pages;
    while ((1 << p.page_shift) < page_size) ++p.page_shift;
    p.rot = rotary ? rot : 0, p.max_pos = max_pos, p.interleaved = interleaved;
    // whole 16-byte accesses everywhere: sizes, strides and addresses allow them
    bool units = D % 16 == 0 && p.rot % 16 == 0;
    for (const Strides *st : {&p.qs, &p.ks, &p.vs}) units = units && !((st->b | st->n | st->h) & 7);
    for (const void *x : {q, k, v, static_cast<const void *>(k_cache), static_cast<const void *>(v_cache),
                          static_cast<const void *>(out_q), static_cast<const void *>(rotary)})
        units = units && !misaligned(x, 16);
    int64_t grid = 0;
    if (q || k) {
        if (units) {
            const int groups = (q ? (Hq + kHeads - 1) / kHeads : 0) + (k ? 2 * ((Hkv + kHeads - 1) / kHeads) : 0);
            const int64_t per = int64_t(groups) * (D / 16);          // threads of a token
            if (per > INT32_MAX / kThreads) return LOOKUP_DRAFT_EINVAL;
            p.tokens = per < kThreads ? int32_t(kThreads / per) : 1;
            grid = (int64_t(B) * N + p.tokens - 1) / p.tokens;
        } else {
            const int64_t heads = (q ? int64_t(Hq) : 0) + (k ? 2 * int64_t(Hkv) : 0);
            grid = (int64_t(B) * N * heads * ((D + 1) / 2) + kThreads - 1) / kThreads;
        }
    }
    const int64_t all = grid + (status ? (int64_t(B) + kThreads / 32 - 1) / (kThreads / 32) : 0);
    if (all > INT32_MAX) return LOOKUP_DRAFT_EINVAL;
    if (all == 0) return LOOKUP_DRAFT_OK;
    p.grid = int32_t(grid);
    const bool half = type == LOOKUP_TYPE_F16;
    auto kernel = units ? (interleaved ? (half ? append_units_kernel<__half, true> : append_units_kernel<__nv_bfloat16, true>)
                                       : (half ? append_units_kernel<__half, false> : append_units_kernel<__nv_bfloat16, false>))
                        : (half ? append_pairs_kernel<__half> : append_pairs_kernel<__nv_bfloat16>);
    return launch_pdl(kernel, unsigned(all), unsigned(kThreads), stream, p);
}

}  // extern "C"
