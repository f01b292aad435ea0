// lookup_norm_append.cu -- norms of query and key heads, rotary positions of a tree's
// nodes, and the append to the paged cache, in one pass.
//
// The contract is in include/lookup_tree.h (lookup_norm_append).
//
// The mathematics: a head x of D elements becomes x_j w_j / sqrt(sum x^2 / D + eps), then
// its pairs are turned, a' = a cos - b sin, b' = b cos + a sin.  Everything in float32;
// the one rounding is the result's, to the tensors' type.
//
// What bounds it: the bytes of q, k and v, read once and written once, and for larger heads the
// instructions around them: 4 prompts of 8191 tokens, 32 and 8 heads of 128, take 231 us
// (3.3 TB/s) with the issue slots 65% busy, half of a CTA empty in its second round of a token's
// 384 threads, and 48 to 72 bytes of a thread's state spilled.  The norm needs the whole head
// before its first element can be written, so the head stays in registers: a thread holds a unit
// of 16 elements (for a rotated unit, 8 pairs that share 8 angles) of one or two heads, the
// D / 16 threads of a head are neighbours in a warp, and the sum of squares is exchanged by
// shuffles.  The angles and weights are read once for a thread's heads.
//
// A head that is no power of two of units (D = 80, 96), a rotated part that is no multiple
// of 16 elements, and strides or addresses that are no multiples of 16 bytes take a
// kernel with a warp per head and a pair per lane and step: right for every case, and slow, with
// 2-byte accesses and every head read twice (those prompts with heads of 80: 688 us, and 597 with
// 40 of 128 elements rotated; 64 trees of up to 63, 14 and 2 heads of 80: 31 us, of 64: 8.1).

#include "lookup_draft.h"
#include "lookup_tree.h"
#include "common.cuh"

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

namespace {

using lkd::allow_dependent_launch;
using lkd::launch_pdl;
using lkd::wait_for_prerequisite_grid;

constexpr int kThreads = 256;
// CTAs per SM for a thread's heads.  4 prompts of 8191 tokens, 32 and 8 heads of 128: 270 us
// with two heads and two CTAs, 254 and 334 with three and four; with one head 265, 233 and 353
// with three, four and five.  (Three CTAs of two heads: 68 us for 62, where 4 prompts have 14
// and 2 heads of 64.)
constexpr int ctas_for(int heads) { return heads == 2 ? 2 : 4; }
constexpr int kFewTokens = 608;          // four for each of 152 SMs
constexpr int kMaxD = 1024;

struct Strides {
    int64_t b, n, h;
};

struct Params {
    const void *q, *k, *v;
    Strides qs, ks, vs;
    const int32_t *kv_len, *q_len, *table, *depth;
    const void *q_weight, *k_weight;
    const float *rotary;
    void *k_cache, *v_cache, *out_q;
    int32_t *status;
    int32_t B, N, Hq, Hkv, D, max_pages, pages, page_shift, rot, max_pos, interleaved;
    float eps;
    int32_t tokens;                      // of a CTA of units_kernel
    int32_t grid;                        // CTAs that append; the ones after them report
};

__device__ inline float to_f32(__half x) { return __half2float(x); }
__device__ inline float to_f32(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ inline void from_f32(float x, __half &y) { y = __float2half_rn(x); }
__device__ inline void from_f32(float x, __nv_bfloat16 &y) { y = __float2bfloat16_rn(x); }

__device__ inline int32_t block_tokens(const Params &p, int b) {
    return p.q_len ? min(max(p.q_len[b], 0), p.N) : p.N;
}

// Where token i of request b is rotated (-1: nowhere) and cached: the first row of its page
// for kv head 0, plus its row in the page, or -1 where the token has no slot.
struct Spot {
    int64_t angle, slot;
};
__device__ inline Spot spot_of(const Params &p, int b, int i) {
    const int64_t kv = max(p.kv_len[b], 0), pos = kv + i, at = pos >> p.page_shift;
    Spot s{0, -1};
    if (p.rotary) {
        s.angle = kv + (p.depth ? p.depth[int64_t(b) * p.N + i] : i);
        if (s.angle < 0 || s.angle >= p.max_pos) return s;
    }
    if (i >= block_tokens(p, b) || at >= p.max_pages) return s;
    const int32_t page = p.table[int64_t(b) * p.max_pages + at];
    if (page >= 0 && page < p.pages)
        s.slot = ((int64_t(page) * p.Hkv) << p.page_shift) + (pos & ((int64_t(1) << p.page_shift) - 1));
    return s;
}

// status, by the CTAs after the appending ones: a warp per request.
__device__ inline void report(const Params &p) {
    const int lane = threadIdx.x & 31;
    const int64_t b = int64_t(blockIdx.x - p.grid) * (kThreads / 32) + (threadIdx.x >> 5);
    if (b >= p.B) return;
    const int n = block_tokens(p, int(b));
    const int64_t first = max(p.kv_len[b], 0);
    bool bad = false;
    if (n > 0)                                           // each page that the block's tokens touch
        for (int64_t at = (first >> p.page_shift) + lane; at <= ((first + n - 1) >> p.page_shift); at += 32) {
            const int32_t page = at < p.max_pages ? p.table[b * p.max_pages + at] : -1;
            bad |= page < 0 || page >= p.pages;
        }
    if (p.rotary) {
        if (!p.depth) bad |= n > 0 && first + n > p.max_pos;
        else
            for (int i = lane; i < n; i += 32) {
                const int64_t angle = first + p.depth[b * p.N + i];
                bad |= angle < 0 || angle >= p.max_pos;
            }
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
__device__ inline uint32_t word(const uint4 &v, int k) { return k == 0 ? v.x : k == 1 ? v.y : k == 2 ? v.z : v.w; }

template <typename T>
__device__ inline void unpack8(const uint4 &v, float *x) {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const float2 f = unpack2(word(v, k), T());
        x[2 * k] = f.x;
        x[2 * k + 1] = f.y;
    }
}
template <typename T>
__device__ inline uint4 pack8(const float *x) {
    return make_uint4(pack2(x[0], x[1], T()), pack2(x[2], x[3], T()), pack2(x[4], x[5], T()), pack2(x[6], x[7], T()));
}

// A pair turned.  Which product each sum takes unrounded is spelled out (as the append without
// a norm has it, but for bfloat16 in neighbours), so that a token's bits do not depend on how many
// come with it.
__device__ inline void turn(float &a, float &b, float c, float s) {
    const float x = a, y = b;
    a = fmaf(x, c, -(y * s));
    b = fmaf(x, s, y * c);
}

// A thread's 16 elements of a head are x[0 .. 8) and x[8 .. 16), from its elements e0 and
// e1 on.  Halves: x[j] pairs with x[8 + j].  Interleaved: x[2 j] with x[2 j + 1].
template <typename T, bool INTER, int kHeads>
__global__ void __launch_bounds__(kThreads, ctas_for(kHeads)) units_kernel(const __grid_constant__ Params p) {
    wait_for_prerequisite_grid();
    allow_dependent_launch();
    if (int(blockIdx.x) >= p.grid) return report(p);
    const uint32_t units = p.D / 16;                     // a power of two, 32 at most
    const int shift = __ffs(int(units)) - 1;
    const float inv_d = 1.0f / float(p.D);               // (exact)
    const int q_groups = p.q ? (p.Hq + kHeads - 1) / kHeads : 0, k_groups = p.k ? (p.Hkv + kHeads - 1) / kHeads : 0;
    const uint32_t per = units * (q_groups + 2 * k_groups);          // threads of a token
    const uint32_t tok0 = blockIdx.x * uint32_t(p.tokens);
    const int b0 = int(tok0 / uint32_t(p.N)), i0 = int(tok0 - uint32_t(b0) * uint32_t(p.N));
    const uint32_t count = p.tokens * per;
    for (uint32_t x0 = threadIdx.x & ~31u; x0 < count; x0 += kThreads) {     // a warp at a time: its lanes stay together
        const uint32_t x = x0 + (threadIdx.x & 31);
        const uint32_t t = x / per, rest = x - t * per;
        int g = int(rest >> shift);
        const int u = int(rest & (units - 1));             // neighbouring threads: neighbouring units of a head
        int b = b0, i = i0 + int(t);
        for (; i >= p.N; i -= p.N) ++b;
        const bool there = x < count && b < p.B;
        const bool is_q = g < q_groups, is_k = !is_q && g < q_groups + k_groups;
        if (!is_q) g -= is_k ? q_groups : q_groups + k_groups;
        const int h0 = g * kHeads, heads = there ? min(kHeads, (is_q ? p.Hq : p.Hkv) - h0) : 0;
        const bool turned = u < p.rot / 16 && (is_q || is_k);
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
        for (int k = 0; k < kHeads; ++k) {
            v0[k] = v1[k] = make_uint4(0, 0, 0, 0);
            if (k < heads) {
                v0[k] = __ldcs(reinterpret_cast<const uint4 *>(src + k * st.h + e0));
                v1[k] = __ldcs(reinterpret_cast<const uint4 *>(src + k * st.h + e1));
            }
        }
        const T *weight = static_cast<const T *>(is_q ? p.q_weight : is_k ? p.k_weight : nullptr);
        uint4 w0 = make_uint4(0, 0, 0, 0), w1 = w0;
        if (weight) {
            w0 = *reinterpret_cast<const uint4 *>(weight + e0);
            w1 = *reinterpret_cast<const uint4 *>(weight + e1);
        }
        const Spot spot = there ? spot_of(p, b, i) : Spot{0, -1};
        float sum[kHeads];
#pragma unroll
        for (int k = 0; k < kHeads; ++k) {
            float a[16];
            unpack8<T>(v0[k], a);
            unpack8<T>(v1[k], a + 8);
            sum[k] = 0.0f;
#pragma unroll
            for (int j = 0; j < 16; ++j) sum[k] = fmaf(a[j], a[j], sum[k]);
        }
        for (uint32_t d = units / 2; d; d >>= 1)
#pragma unroll
            for (int k = 0; k < kHeads; ++k) sum[k] += __shfl_xor_sync(0xffffffffu, sum[k], int(d));
        if (!there) continue;
        T *dst;
        int64_t step;
        if (is_q) {
            dst = static_cast<T *>(p.out_q) + ((int64_t(b) * p.N + i) * p.Hq + h0) * p.D;
            step = p.D;
        } else {
            if (spot.slot < 0) continue;
            dst = static_cast<T *>(is_k ? p.k_cache : p.v_cache) + (spot.slot + (int64_t(h0) << p.page_shift)) * p.D;
            step = int64_t(p.D) << p.page_shift;
        }
        if (spot.slot < 0) {                             // a query row past the block, or without a slot
#pragma unroll
            for (int k = 0; k < kHeads; ++k) v0[k] = v1[k] = make_uint4(0, 0, 0, 0);
        } else if (weight || turned) {
            float c[8], s[8], w[16];
            if (turned) {
                const float *row = p.rotary + spot.angle * p.rot + 8 * u;
#pragma unroll
                for (int j = 0; j < 8; j += 4) {
                    *reinterpret_cast<float4 *>(c + j) = *reinterpret_cast<const float4 *>(row + j);
                    *reinterpret_cast<float4 *>(s + j) = *reinterpret_cast<const float4 *>(row + p.rot / 2 + j);
                }
            }
            unpack8<T>(w0, w);
            unpack8<T>(w1, w + 8);
#pragma unroll
            for (int k = 0; k < kHeads; ++k) {
                float a[16];
                unpack8<T>(v0[k], a);
                unpack8<T>(v1[k], a + 8);
                if (weight) {
                    const float r = rsqrtf(fmaf(sum[k], inv_d, p.eps));
#pragma unroll
                    for (int j = 0; j < 16; ++j) a[j] *= r * w[j];
                }
                if (turned) {
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        float &f = a[INTER ? 2 * j : j], &h = a[INTER ? 2 * j + 1 : 8 + j];
                        turn(f, h, c[j], s[j]);
                    }
                }
                v0[k] = pack8<T>(a);
                v1[k] = pack8<T>(a + 8);
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

// A warp per head of a token.
template <typename T>
__global__ void __launch_bounds__(kThreads) heads_kernel(const __grid_constant__ Params p) {
    wait_for_prerequisite_grid();
    allow_dependent_launch();
    if (int(blockIdx.x) >= p.grid) return report(p);
    const int lane = threadIdx.x & 31;
    const int heads = (p.q ? p.Hq : 0) + (p.k ? 2 * p.Hkv : 0);
    const int64_t head_id = int64_t(blockIdx.x) * (kThreads / 32) + (threadIdx.x >> 5);
    const int64_t tok = head_id / heads;
    int h = int(head_id - tok * heads);
    const int b = int(tok / p.N), i = int(tok - int64_t(b) * p.N);
    if (b >= p.B) return;
    const bool is_q = p.q && h < p.Hq;
    const Spot spot = spot_of(p, b, i);
    if (!is_q && spot.slot < 0) return;
    const T *src, *weight = nullptr;
    T *dst;
    bool rotate = p.rotary != nullptr;
    if (is_q) {
        src = static_cast<const T *>(p.q) + b * p.qs.b + i * p.qs.n + h * p.qs.h;
        dst = static_cast<T *>(p.out_q) + (tok * p.Hq + h) * p.D;
        weight = static_cast<const T *>(p.q_weight);
    } else {
        if (p.q) h -= p.Hq;
        const bool is_k = h < p.Hkv;
        if (!is_k) h -= p.Hkv;
        const Strides &st = is_k ? p.ks : p.vs;
        src = static_cast<const T *>(is_k ? p.k : p.v) + b * st.b + i * st.n + h * st.h;
        dst = static_cast<T *>(is_k ? p.k_cache : p.v_cache) + (spot.slot + (int64_t(h) << p.page_shift)) * p.D;
        if (is_k) weight = static_cast<const T *>(p.k_weight);
        rotate = rotate && is_k;
    }
    T zero;
    from_f32(0.0f, zero);
    if (spot.slot < 0) {                                 // a query row past the block, or without a slot
        for (int j = lane; j < p.D; j += 32) dst[j] = zero;
        return;
    }
    float r = 1.0f;
    if (weight) {
        float sum = 0.0f;
        for (int j = lane; j < p.D; j += 32) {
            const float x = to_f32(src[j]);
            sum = fmaf(x, x, sum);
        }
#pragma unroll
        for (int d = 16; d; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
        r = rsqrtf(sum / float(p.D) + p.eps);
    }
    const int half = rotate ? p.rot / 2 : 0;
    auto scaled = [&](int j) { return weight ? to_f32(src[j]) * (r * to_f32(weight[j])) : to_f32(src[j]); };
    for (int e = lane; e < half; e += 32) {
        const int j0 = p.interleaved ? 2 * e : e, j1 = p.interleaved ? 2 * e + 1 : e + half;
        const float *row = p.rotary + spot.angle * p.rot;
        const float c = row[e], s = row[half + e];
        float x = scaled(j0), y = scaled(j1);
        turn(x, y, c, s);
        from_f32(x, dst[j0]);
        from_f32(y, dst[j1]);
    }
    for (int j = 2 * half + lane; j < p.D; j += 32) {
        if (weight) from_f32(scaled(j), dst[j]);
        else dst[j] = src[j];
    }
}

// Heads of a thread of units_kernel, for `per` threads a token with one.  Many tokens: two of up
// to 64 elements share what their thread reads and works out (us, two and one: 64 trees of 63,
// 14 and 2 heads of 64, 7.6 and 8.8; 1024 of 64 116 and 119; 4 prompts of 8191 62 and 66; 14 and
// 2 of 32 34 and 35; but 16 and 16 of 64 145 and 143), larger ones want the warps more (32 and 8
// heads of 128, the same batches: 32.8 and 31.8, 530 and 468, 287 and 256; 16 and 4 of 256: 34
// and 33, 545 and 479, 291 and 259).  Few tokens, all at once on the device: one head, the
// shorter way (one tree of 15, 14 and 2 heads of 64: 3.4 and 2.8; 8 of 32: 3.6 and 3.0), unless a
// CTA would have to go round twice for a token (32 and 8 heads of 128: 2.8 and 3.8; 3.2 and 4.4;
// 512 single tokens 5.4 and 5.9; 504 with 64 and 8 heads 8.7 and 8.5).
int heads_for(int64_t tokens, int64_t per, int D) {
    if (tokens <= kFewTokens) return per > kThreads ? 2 : 1;
    return D <= 64 ? 2 : 1;
}

template <typename T>
auto units_for(bool interleaved, int heads) {
    if (heads == 2) return interleaved ? units_kernel<T, true, 2> : units_kernel<T, false, 2>;
    return interleaved ? units_kernel<T, true, 1> : units_kernel<T, false, 1>;
}

bool misaligned(const void *p, size_t to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) != 0; }

}  // namespace

extern "C" {

int lookup_norm_append(const void *q, const int64_t *q_strides, const void *k, const int64_t *k_strides,
                       const void *v, const int64_t *v_strides, const int32_t *kv_len, const int32_t *q_len,
                       const int32_t *block_table, int32_t B, int32_t N, int32_t Hq, int32_t Hkv, int32_t D,
                       int32_t max_pages, int32_t pages, int32_t page_size, const void *q_weight,
                       const void *k_weight, float eps, const float *rotary, int32_t rot, int32_t max_pos,
                       const int32_t *depth, int32_t interleaved, int32_t type, void *k_cache, void *v_cache,
                       void *out_q, int32_t *status, struct CUstream_st *stream) {
    lkd::TraceRange trace_("lookup_norm_append");
    if (B < 0 || N < 0 || Hq < 0 || Hkv < 1 || D < 1 || D > kMaxD || max_pages < 1 || pages < 1 || page_size < 1 ||
        (page_size & (page_size - 1)) || (q && Hq < 1) || !(eps >= 0.0f && eps < INFINITY))
        return LOOKUP_DRAFT_EINVAL;
    if (rotary && (rot < 2 || rot > D || (rot & 1) || max_pos < 1)) return LOOKUP_DRAFT_EINVAL;
    if (type != LOOKUP_TYPE_F16 && type != LOOKUP_TYPE_BF16) return LOOKUP_DRAFT_EINVAL;
    if (B == 0 || N == 0) return LOOKUP_DRAFT_OK;
    if (int64_t(B) * N > INT32_MAX) return LOOKUP_DRAFT_EINVAL;
    if (!kv_len || !block_table || !k != !v || (k && (!k_cache || !v_cache || !k_strides || !v_strides)) ||
        (q && (!out_q || !q_strides)))
        return LOOKUP_DRAFT_EINVAL;
    for (const void *x : {q, k, v, static_cast<const void *>(k_cache), static_cast<const void *>(v_cache),
                          static_cast<const void *>(out_q), q_weight, k_weight})
        if (misaligned(x, 2)) return LOOKUP_DRAFT_EINVAL;
    for (const void *x : {static_cast<const void *>(kv_len), static_cast<const void *>(q_len),
                          static_cast<const void *>(block_table), static_cast<const void *>(rotary),
                          static_cast<const void *>(depth), static_cast<const void *>(status)})
        if (misaligned(x, 4)) return LOOKUP_DRAFT_EINVAL;
    Params p{};
    p.q = q, p.k = k, p.v = v;
    auto strides = [&](const int64_t *s, int32_t heads) {    // an axis of one has any: it is not used
        return Strides{B > 1 ? s[0] : 0, N > 1 ? s[1] : 0, heads > 1 ? s[2] : 0};
    };
    if (q) p.qs = strides(q_strides, Hq);
    if (k) p.ks = strides(k_strides, Hkv);
    if (v) p.vs = strides(v_strides, Hkv);
    p.kv_len = kv_len, p.q_len = q_len, p.table = block_table, p.depth = depth, p.rotary = rotary;
    p.q_weight = q_weight, p.k_weight = k_weight, p.eps = eps;
    p.k_cache = k_cache, p.v_cache = v_cache, p.out_q = out_q, p.status = status;
    p.B = B, p.N = N, p.Hq = Hq, p.Hkv = Hkv, p.D = D, p.max_pages = max_pages, p.pages = pages;
    while ((1 << p.page_shift) < page_size) ++p.page_shift;
    p.rot = rotary ? rot : 0, p.max_pos = max_pos, p.interleaved = interleaved;
    // whole 16-byte accesses everywhere, and heads that divide a warp
    bool units = D % 16 == 0 && D <= 512 && (D & (D - 1)) == 0 && p.rot % 16 == 0;
    for (const Strides *st : {&p.qs, &p.ks, &p.vs}) units = units && !((st->b | st->n | st->h) & 7);
    for (const void *x : {q, k, v, static_cast<const void *>(k_cache), static_cast<const void *>(v_cache),
                          static_cast<const void *>(out_q), static_cast<const void *>(rotary), q_weight, k_weight})
        units = units && !misaligned(x, 16);
    int64_t grid = 0;
    int each = 1;                                        // heads of a thread of units_kernel
    if (q || k) {
        if (units) {
            const int64_t heads = (q ? int64_t(Hq) : 0) + (k ? 2 * int64_t(Hkv) : 0);
            each = heads_for(int64_t(B) * N, heads * (D / 16), D);
            const int64_t groups = (q ? (int64_t(Hq) + each - 1) / each : 0) + (k ? 2 * ((int64_t(Hkv) + each - 1) / each) : 0);
            const int64_t per = groups * (D / 16);       // threads of a token
            if (per > INT32_MAX / kThreads) return LOOKUP_DRAFT_EINVAL;
            p.tokens = per < kThreads ? int32_t(kThreads / per) : 1;
            grid = (int64_t(B) * N + p.tokens - 1) / p.tokens;
        } else {
            const int64_t heads = (q ? int64_t(Hq) : 0) + (k ? 2 * int64_t(Hkv) : 0);
            if (heads > INT32_MAX) return LOOKUP_DRAFT_EINVAL;
            grid = (int64_t(B) * N * heads + kThreads / 32 - 1) / (kThreads / 32);
        }
    }
    const int64_t all = grid + (status ? (int64_t(B) + kThreads / 32 - 1) / (kThreads / 32) : 0);
    if (all > INT32_MAX) return LOOKUP_DRAFT_EINVAL;
    if (all == 0) return LOOKUP_DRAFT_OK;
    p.grid = int32_t(grid);
    const bool half = type == LOOKUP_TYPE_F16;
    auto kernel = !units ? (half ? heads_kernel<__half> : heads_kernel<__nv_bfloat16>)
                         : half ? units_for<__half>(interleaved, each) : units_for<__nv_bfloat16>(interleaved, each);
    return launch_pdl(kernel, unsigned(all), unsigned(kThreads), stream, p);
}

}  // extern "C"
