// lookup_logits.cu -- verification of proposal blocks against the target's logits.
//
// The contract is in include/lookup_target.h (lookup_verify_logits).  Two kernels:
// stats_kernel reads every row of logits once and leaves, per row segment, the
// running maximum m, s = sum exp((x - m) / T) and the lowest index of m;
// pick_kernel joins a request's segments, finds its first rejected position and
// draws that row's token.

#include "lookup_draft.h"
#include "lookup_target.h"
#include "common.cuh"

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cfloat>
#include <cmath>
#include <cstdint>

namespace {

using lkd::allow_dependent_launch;
using lkd::kMaxBlock;
using lkd::launch_pdl;
using lkd::wait_for_prerequisite_grid;

constexpr int kStatThreads = 256;
constexpr int kPickThreads = 512;
constexpr int kMaxSegs = 64;             // segments of a row at most
constexpr int kMaxV = 1 << 30;

struct Params {
    const int32_t *block, *len;
    const void *logits;
    int64_t lb, lp;                      // strides of logits: request, position (elements)
    const float *noise, *temperature, *u, *qprobs;
    int64_t qb, qp;                      // strides of qprobs
    const int32_t *point_mass;
    int32_t B, P, V, segs;
    int32_t *out_accepted, *out_commit, *out_ncommit;
    float *out_logprobs;
    float4 *part;                        // [B][P + 1][segs]: m, s, index of m (bits), unused
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

__device__ inline Stat warp_join(Stat v, float inv_t) {
#pragma unroll
    for (int d = 16; d; d >>= 1) {
        Stat o;
        o.m = __shfl_xor_sync(0xffffffffu, v.m, d);
        o.s = __shfl_xor_sync(0xffffffffu, v.s, d);
        o.at = __shfl_xor_sync(0xffffffffu, v.at, d);
        v = join(v, o, inv_t);
    }
    return v;
}

template <typename T>
__global__ void __launch_bounds__(kStatThreads) stats_kernel(Params p) {
    __shared__ Stat warp_stat[kStatThreads / 32];
    wait_for_prerequisite_grid();
    allow_dependent_launch();
    const int seg = blockIdx.x % p.segs;
    const int64_t row_id = blockIdx.x / p.segs;
    const int b = int(row_id / (p.P + 1)), i = int(row_id % (p.P + 1));
    const int n = p.len[b];
    if (i > n || n > p.P) return;                       // a row no proposal is tested in
    const T *row = static_cast<const T *>(p.logits) + b * p.lb + i * p.lp;
    const float inv_t = inv_temperature(p, b);
    const int lo = int(int64_t(p.V) * seg / p.segs), hi = int(int64_t(p.V) * (seg + 1) / p.segs);
    Stat v{-INFINITY, 0.0f, INT32_MAX};
    for (int j = lo + threadIdx.x; j < hi; j += kStatThreads) {
        const float x = logit(row, j);
        if (x > v.m) {
            v.s = v.m == -INFINITY ? 1.0f : v.s * weight(v.m, x, inv_t) + 1.0f;
            v.m = x;
            v.at = j;
        } else if (x != -INFINITY) {
            v.s += weight(x, v.m, inv_t);
        }
    }
    v = warp_join(v, inv_t);
    if ((threadIdx.x & 31) == 0) warp_stat[threadIdx.x >> 5] = v;
    __syncthreads();
    if (threadIdx.x < 32) {
        v = threadIdx.x < kStatThreads / 32 ? warp_stat[threadIdx.x] : Stat{-INFINITY, 0.0f, INT32_MAX};
        v = warp_join(v, inv_t);
        if (threadIdx.x == 0) p.part[row_id * p.segs + seg] = make_float4(v.m, v.s, __int_as_float(v.at), 0.0f);
    }
}

// Row (b, i)'s statistics from its segments, by one warp (every lane gets them).
__device__ inline Stat row_stat(const Params &p, int b, int i, float inv_t, int lane) {
    const float4 *part = p.part + (int64_t(b) * (p.P + 1) + i) * p.segs;
    Stat v{-INFINITY, 0.0f, INT32_MAX};
    for (int k = lane; k < p.segs; k += 32) {
        const float4 q = part[k];
        v = join(v, Stat{q.x, q.y, __float_as_int(q.z)}, inv_t);
    }
    return warp_join(v, inv_t);
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

// One CTA per request.
template <typename T>
__global__ void __launch_bounds__(kPickThreads) pick_kernel(Params p) {
    __shared__ int s_first;
    __shared__ Stat s_row;
    __shared__ Best warp_res[kPickThreads / 32], warp_all[kPickThreads / 32];
    wait_for_prerequisite_grid();
    allow_dependent_launch();
    const int b = blockIdx.x, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int P = p.P, n = p.len[b];
    int32_t *commit = p.out_commit + int64_t(b) * (P + 1);
    float *lps = p.out_logprobs ? p.out_logprobs + int64_t(b) * (P + 1) : nullptr;
    if (n < 0 || n > P) {                               // no valid block: an error row
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
    const float inv_t = inv_temperature(p, b);
    const T *rows = static_cast<const T *>(p.logits) + b * p.lb;
    const int32_t *block = p.block + int64_t(b) * P;
    if (tid == 0) s_first = n;
    __syncthreads();
    // a warp per position: is its proposal accepted, and with which probability
    for (int i = warp; i < n; i += kPickThreads / 32) {
        const Stat v = row_stat(p, b, i, inv_t, lane);
        const int d = block[i];
        const bool fits = d >= 0 && d < p.V && v.m > -INFINITY;
        const float x = fits ? logit(rows + i * p.lp, d) : -INFINITY;
        bool ok;
        if (greedy) {
            ok = fits && d == v.at;
        } else {
            const float pd = fits ? weight(x, v.m, inv_t) / v.s : 0.0f;
            const bool point = !p.qprobs || (p.point_mass && p.point_mass[int64_t(b) * P + i] != 0);
            const float q = point || !fits ? 1.0f : p.qprobs[b * p.qb + i * p.qp + d];
            ok = __fmul_rn(p.u[int64_t(b) * P + i], q) < pd;
        }
        if (lane == 0) {
            if (!ok) atomicMin(&s_first, i);
            if (lps) lps[i] = ok ? (x == v.m ? 0.0f : (x - v.m) * inv_t) - logf(v.s) : 0.0f;
        }
    }
    __syncthreads();
    const int a = s_first;
    if (warp == 0) {
        const Stat v = row_stat(p, b, a, inv_t, lane);
        if (lane == 0) s_row = v;
    }
    __syncthreads();
    const Stat row = s_row;
    const T *x = rows + a * p.lp;
    int32_t token = row.m > -INFINITY ? row.at : -1;
    if (!greedy && token >= 0) {
        // the race: the residual's best key, and p's own for a residual of nothing
        const bool rejected = a < n;
        const bool point = !p.qprobs || (p.point_mass && rejected && p.point_mass[int64_t(b) * P + a] != 0);
        const int32_t d = rejected && point ? block[a] : -1;
        const float *q = rejected && !point ? p.qprobs + b * p.qb + a * p.qp : nullptr;
        const float *noise = p.noise + int64_t(b) * p.V;
        Best res{-1.0f, INT32_MAX}, all{-1.0f, INT32_MAX};
        for (int j = tid; j < p.V; j += kPickThreads) {
            const float pj = weight(logit(x, j), row.m, inv_t) / row.s, e = noise[j];
            const float left = j == d ? 0.0f : (q ? pj - q[j] : pj);
            if (left > 0.0f) res = better(res, Best{left / e, j});
            if (pj > 0.0f) all = better(all, Best{pj / e, j});
        }
        res = warp_better(res);
        all = warp_better(all);
        if (lane == 0) {
            warp_res[warp] = res;
            warp_all[warp] = all;
        }
        __syncthreads();
        if (warp == 0) {
            res = lane < kPickThreads / 32 ? warp_res[lane] : Best{-1.0f, INT32_MAX};
            all = lane < kPickThreads / 32 ? warp_all[lane] : Best{-1.0f, INT32_MAX};
            res = warp_better(res);
            all = warp_better(all);
            token = res.key >= 0.0f ? res.at : all.at;
        }
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

int segments(int32_t B, int32_t P, int32_t V) {
    const int64_t rows = int64_t(B) * (P + 1);
    int64_t s = 152 * 16 / (rows > 0 ? rows : 1) + 1;
    const int64_t most = (int64_t(V) + 4095) / 4096;
    if (s > most) s = most;
    return int(s > kMaxSegs ? kMaxSegs : s);
}

template <typename T>
int launch(const Params &p, cudaStream_t stream) {
    int rc = launch_pdl(stats_kernel<T>, unsigned(int64_t(p.B) * (p.P + 1) * p.segs), unsigned(kStatThreads), stream, p);
    if (rc != LOOKUP_DRAFT_OK) return rc;
    return launch_pdl(pick_kernel<T>, unsigned(p.B), unsigned(kPickThreads), stream, p);
}

bool misaligned(const void *p, size_t to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) != 0; }

}  // namespace

extern "C" {

size_t lookup_verify_logits_workspace_bytes(int32_t B, int32_t P, int32_t V) {
    if (B < 0 || P < 0 || P > kMaxBlock || V < 1 || V >= kMaxV) return 0;
    return size_t(B) * size_t(P + 1) * size_t(segments(B, P, V)) * sizeof(float4) + 16;
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
    const int segs = segments(B, P, V);
    if (int64_t(B) * (P + 1) * segs > INT32_MAX) return LOOKUP_DRAFT_EINVAL;
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
    Params p{block, len, logits, logits_strides[0], logits_strides[1], noise, noise ? temperature : nullptr, u,
             with_q ? qprobs : nullptr, with_q ? qprobs_strides[0] : 0, with_q ? qprobs_strides[1] : 0, point_mass,
             B, P, V, segs, out_accepted, out_commit, out_ncommit, out_logprobs, static_cast<float4 *>(workspace)};
    if (type == LOOKUP_TYPE_F32) return launch<float>(p, stream);
    if (type == LOOKUP_TYPE_F16) return launch<__half>(p, stream);
    return launch<__nv_bfloat16>(p, stream);
}

}  // extern "C"
