// lookup_kv_append.cu -- rotary positions and the append to the paged cache.
//
// The contract is in include/lookup_target.h (lookup_kv_append).  One kernel, one
// thread per (token, head, rotated pair or copied pair of elements).

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

// 1 where any of the request's tokens has no slot, by its whole block of threads.
__global__ void status_kernel(Params p) {
    wait_for_prerequisite_grid();
    allow_dependent_launch();
    const int b = blockIdx.x;
    const int n = block_tokens(p, b);
    bool bad = false;
    for (int i = threadIdx.x; i < n; i += blockDim.x) bad |= slot_of(p, b, int64_t(max(p.kv_len[b], 0)) + i) < 0;
    bad = __syncthreads_or(bad) != 0;
    if (threadIdx.x == 0) p.status[b] = bad ? 1 : 0;
}

template <typename T>
__global__ void __launch_bounds__(kThreads) append_kernel(Params p) {
    wait_for_prerequisite_grid();
    allow_dependent_launch();
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
    if (q) p.qs = Strides{q_strides[0], q_strides[1], q_strides[2]};
    if (k) p.ks = Strides{k_strides[0], k_strides[1], k_strides[2]};
    if (v) p.vs = Strides{v_strides[0], v_strides[1], v_strides[2]};
    p.kv_len = kv_len, p.q_len = q_len, p.table = block_table, p.rotary = rotary;
    p.k_cache = k_cache, p.v_cache = v_cache, p.out_q = out_q, p.status = status;
    p.B = B, p.N = N, p.Hq = Hq, p.Hkv = Hkv, p.D = D, p.max_pages = max_pages, p.pages = pages;
    while ((1 << p.page_shift) < page_size) ++p.page_shift;
    p.rot = rotary ? rot : 0, p.max_pos = max_pos, p.interleaved = interleaved;
    if (q || k) {
        const int64_t threads = int64_t(B) * N * ((q ? Hq : 0) + (k ? 2 * Hkv : 0)) * ((D + 1) / 2);
        const int64_t grid = (threads + kThreads - 1) / kThreads;
        if (grid > INT32_MAX) return LOOKUP_DRAFT_EINVAL;
        const int rc = type == LOOKUP_TYPE_F16
                           ? launch_pdl(append_kernel<__half>, unsigned(grid), unsigned(kThreads), stream, p)
                           : launch_pdl(append_kernel<__nv_bfloat16>, unsigned(grid), unsigned(kThreads), stream, p);
        if (rc != LOOKUP_DRAFT_OK) return rc;
    }
    if (status) return launch_pdl(status_kernel, unsigned(B), unsigned(kThreads), stream, p);
    return LOOKUP_DRAFT_OK;
}

}  // extern "C"
