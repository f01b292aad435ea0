// lookup_attention.cu -- attention of a verify block over the paged cache.
//
// The contract is in include/lookup_target.h (lookup_paged_attention).  One warp per
// (query row, part of the cache's length), a running maximum and sum; a second
// kernel joins the parts.

#include "lookup_draft.h"
#include "lookup_target.h"
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

constexpr int kWarps = 4;
constexpr int kMaxParts = 32;

struct Params {
    const void *q;
    int64_t qb, qn, qh;
    const void *k_cache, *v_cache;
    const int32_t *table, *kv_len, *q_len;
    int32_t B, N, Hq, Hkv, max_pages, pages, page_shift, window, parts;
    float scale;
    void *out;
    float *lse, *ws;                     // ws: [row][parts][D + 2]: m, s, o
};

__device__ inline float to_f32(__half x) { return __half2float(x); }
__device__ inline float to_f32(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ inline void from_f32(float x, __half &y) { y = __float2half_rn(x); }
__device__ inline void from_f32(float x, __nv_bfloat16 &y) { y = __float2bfloat16_rn(x); }

// Positions [lo, hi) that row (b, i) sees.
__device__ inline void range_of(const Params &p, int b, int i, int64_t &lo, int64_t &hi) {
    const int n = p.q_len ? min(max(p.q_len[b], 0), p.N) : p.N;
    lo = hi = 0;
    if (i >= n) return;
    const int64_t pos = int64_t(max(p.kv_len[b], 0)) + i;
    lo = p.window > 0 ? max(pos - p.window + 1, int64_t(0)) : 0;
    hi = max(min(pos + 1, int64_t(p.max_pages) << p.page_shift), lo);
}

template <typename T, int D>
__global__ void __launch_bounds__(kWarps * 32) part_kernel(Params p) {
    constexpr int E = D / 32;
    wait_for_prerequisite_grid();
    allow_dependent_launch();
    const int lane = threadIdx.x & 31;
    const int64_t id = int64_t(blockIdx.x) * kWarps + (threadIdx.x >> 5);
    const int64_t row = id / p.parts;
    const int part = int(id - row * p.parts);
    if (row >= int64_t(p.B) * p.N * p.Hq) return;
    const int h = int(row % p.Hq);
    const int i = int(row / p.Hq % p.N), b = int(row / p.Hq / p.N);
    const int hk = h / (p.Hq / p.Hkv);
    int64_t lo, hi;
    range_of(p, b, i, lo, hi);
    const int64_t span = hi - lo;
    const int64_t j0 = lo + span * part / p.parts, j1 = lo + span * (part + 1) / p.parts;
    const T *q = static_cast<const T *>(p.q) + b * p.qb + i * p.qn + h * p.qh;
    float qr[E], o[E];
#pragma unroll
    for (int e = 0; e < E; ++e) {
        qr[e] = j1 > j0 ? to_f32(q[lane + 32 * e]) : 0.0f;
        o[e] = 0.0f;
    }
    float m = -INFINITY, s = 0.0f;
    for (int64_t j = j0; j < j1; ++j) {
        const int32_t page = p.table[int64_t(b) * p.max_pages + (j >> p.page_shift)];
        const bool there = page >= 0 && page < p.pages;
        const int64_t at = ((((int64_t(page) * p.Hkv + hk) << p.page_shift) + (j & ((1 << p.page_shift) - 1)))) * D;
        float dot = 0.0f, v[E];
#pragma unroll
        for (int e = 0; e < E; ++e) {
            v[e] = there ? to_f32(static_cast<const T *>(p.v_cache)[at + lane + 32 * e]) : 0.0f;
            dot += there ? qr[e] * to_f32(static_cast<const T *>(p.k_cache)[at + lane + 32 * e]) : 0.0f;
        }
#pragma unroll
        for (int d = 16; d; d >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, d);
        dot *= p.scale;
        const float m2 = fmaxf(m, dot);
        const float f = m == m2 ? 1.0f : expf(m - m2), w = dot == m2 ? 1.0f : expf(dot - m2);
        s = s * f + w;
#pragma unroll
        for (int e = 0; e < E; ++e) o[e] = o[e] * f + w * v[e];
        m = m2;
    }
    float *ws = p.ws + (row * p.parts + part) * (D + 2);
    if (lane == 0) {
        ws[0] = m;
        ws[1] = s;
    }
#pragma unroll
    for (int e = 0; e < E; ++e) ws[2 + lane + 32 * e] = o[e];
}

template <typename T, int D>
__global__ void __launch_bounds__(kWarps * 32) join_kernel(Params p) {
    constexpr int E = D / 32;
    wait_for_prerequisite_grid();
    allow_dependent_launch();
    const int lane = threadIdx.x & 31;
    const int64_t row = int64_t(blockIdx.x) * kWarps + (threadIdx.x >> 5);
    if (row >= int64_t(p.B) * p.N * p.Hq) return;
    const float *ws = p.ws + row * p.parts * (D + 2);
    float m = -INFINITY, s = 0.0f, o[E] = {};
    for (int k = 0; k < p.parts; ++k, ws += D + 2) {
        const float mk = ws[0];
        if (ws[1] == 0.0f) continue;                     // an empty part
        const float m2 = fmaxf(m, mk);
        const float f = m == m2 ? 1.0f : expf(m - m2), w = mk == m2 ? 1.0f : expf(mk - m2);
        s = s * f + w * ws[1];
#pragma unroll
        for (int e = 0; e < E; ++e) o[e] = o[e] * f + w * ws[2 + lane + 32 * e];
        m = m2;
    }
    T *out = static_cast<T *>(p.out) + row * D;
#pragma unroll
    for (int e = 0; e < E; ++e) from_f32(s > 0.0f ? o[e] / s : 0.0f, out[lane + 32 * e]);
    if (lane == 0 && p.lse) p.lse[row] = s > 0.0f ? m + logf(s) : -INFINITY;
}

int parts_for(int64_t rows) {
    const int64_t want = 152 * 64 / (rows > 0 ? rows : 1) + 1;
    return int(want > kMaxParts ? kMaxParts : want);
}

template <typename T, int D>
int launch(const Params &p, cudaStream_t stream) {
    const int64_t rows = int64_t(p.B) * p.N * p.Hq;
    const int rc = launch_pdl(part_kernel<T, D>, unsigned((rows * p.parts + kWarps - 1) / kWarps),
                              unsigned(kWarps * 32), stream, p);
    if (rc != LOOKUP_DRAFT_OK) return rc;
    return launch_pdl(join_kernel<T, D>, unsigned((rows + kWarps - 1) / kWarps), unsigned(kWarps * 32), stream, p);
}

template <typename T>
int launch_d(const Params &p, int D, cudaStream_t stream) {
    return D == 64 ? launch<T, 64>(p, stream) : D == 128 ? launch<T, 128>(p, stream) : launch<T, 256>(p, stream);
}

bool misaligned(const void *p, size_t to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) != 0; }

}  // namespace

extern "C" {

size_t lookup_paged_attention_workspace_bytes(int32_t B, int32_t N, int32_t Hq, int32_t Hkv, int32_t D) {
    if (B < 0 || N < 0 || Hq < 1 || Hkv < 1 || Hq % Hkv || (D != 64 && D != 128 && D != 256)) return 0;
    const int64_t rows = int64_t(B) * N * Hq;
    return size_t(rows) * size_t(parts_for(rows)) * size_t(D + 2) * sizeof(float) + 16;
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
    if (int64_t(pages) * Hkv * page_size > INT32_MAX) return LOOKUP_DRAFT_EINVAL;
    if (B == 0 || N == 0) return LOOKUP_DRAFT_OK;
    const int64_t rows = int64_t(B) * N * Hq;
    if (rows > (int64_t(1) << 30)) return LOOKUP_DRAFT_EINVAL;
    if (!q || !q_strides || !k_cache || !v_cache || !block_table || !kv_len || !out || !workspace)
        return LOOKUP_DRAFT_EINVAL;
    for (const void *x : {q, k_cache, v_cache, static_cast<const void *>(workspace), static_cast<const void *>(out)})
        if (misaligned(x, 16)) return LOOKUP_DRAFT_EINVAL;
    for (int k = 0; k < 3; ++k)
        if (q_strides[k] & 7) return LOOKUP_DRAFT_EINVAL;
    if (misaligned(block_table, 4) || misaligned(kv_len, 4) || misaligned(q_len, 4) || misaligned(lse, 4))
        return LOOKUP_DRAFT_EINVAL;
    if (workspace_bytes < lookup_paged_attention_workspace_bytes(B, N, Hq, Hkv, D)) return LOOKUP_DRAFT_EINVAL;
    Params p{};
    p.q = q, p.qb = q_strides[0], p.qn = q_strides[1], p.qh = q_strides[2];
    p.k_cache = k_cache, p.v_cache = v_cache, p.table = block_table, p.kv_len = kv_len, p.q_len = q_len;
    p.B = B, p.N = N, p.Hq = Hq, p.Hkv = Hkv, p.max_pages = max_pages, p.pages = pages;
    while ((1 << p.page_shift) < page_size) ++p.page_shift;
    p.window = window, p.parts = parts_for(rows), p.scale = scale, p.out = out, p.lse = lse;
    p.ws = static_cast<float *>(workspace);
    return type == LOOKUP_TYPE_F16 ? launch_d<__half>(p, D, stream) : launch_d<__nv_bfloat16>(p, D, stream);
}

}  // extern "C"
