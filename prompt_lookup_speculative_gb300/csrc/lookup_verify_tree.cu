// lookup_verify_tree.cu -- verification of trees of proposals against the target's logits.
//
// The contract is in include/lookup_tree.h (lookup_verify_tree).
//
// The mathematics: at a node with the distribution p its children's tokens take the
// intervals [0, p(t1)), [p(t1), p(t1) + p(t2)), ... of [0, 1), and one uniform number u
// falls into one of them, or past them all.  There the token comes from p without those
// tokens, by a race of exponentials.  Both together draw from p exactly, with one number
// per node and no division by what is left after a refusal.
//
// What bounds it: the logits of the nodes along the branch, each row read once, but which
// rows these are only the rows before them tell.
//
// stats_kernel (logits.cuh) takes every node's row; walk_kernel, a cluster of CTAs per
// request, joins the rows' segments, tests every node against its parent's row, follows
// the branch and draws the last token from its end's row.  64 trees of 32 over 151936 bf16
// logits: 123 us sampled and 132 greedy (which looks for every row's index) for all 622 MB; the
// branches' rows alone are a fifth.  Of 32 such trees the rows take 58 us (5.4 TB/s) and the walks
// 23, with nothing of their noise on the way before them.  One greedy tree of 15 over 32000
// float32 logits: 6.1 us, 12.7 to 15.2 as called.

#include "logits.cuh"

#include "lookup_tree.h"

namespace {

struct TreeParams {
    Params rows;                         // P = N - 1, len = the nodes' count
    const int32_t *parent;
    int32_t *out_path;
};

constexpr int kNodes = LOOKUP_TREE_MAX_NODES;

// A request's tree in shared memory.
struct Tree {
    int32_t token[kNodes], parent[kNodes], next[kNodes], path[kNodes + 1];
    float weight[kNodes];                // p of the token in the parent's row; 0: no one's child, or an earlier one's token
    Stat row[kNodes];
    int32_t kids[kNodes];                // tokens of the last node's children
    int32_t accepted, kid_count;
};

template <typename T>
__global__ void __launch_bounds__(kPickThreads) walk_kernel(const __grid_constant__ TreeParams tp) {
    __shared__ Tree tree;
    __shared__ uint64_t warps[3][kPickThreads / 32], places[3][kMaxCluster];
    const Params &p = tp.rows;
    const int b = blockIdx.x / p.cluster, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int rank = int(cluster_rank());
    const int per = int((uint32_t(p.V) + uint32_t(p.cluster) - 1) / uint32_t(p.cluster));
    const int lo = min(rank * per, p.V), hi = min(lo + per, p.V);    // this CTA's part of the race
    const int N = p.P + 1;
    wait_for_prerequisite_grid();
    allow_dependent_launch();
    const int n = p.len[b];
    const int64_t out = int64_t(b) * N;
    float *lps = p.out_logprobs ? p.out_logprobs + out : nullptr;
    // no valid tree, or logits that did not arrive in time: an error row
    bool bad = tid < p.ctas && p.status[tid] != 0;
    static_assert(kMaxCtas <= kPickThreads, "a thread per CTA of stats_kernel");
    if (__syncthreads_or(bad || n < 1 || n > N)) {
        if (rank) return;
        for (int i = tid; i < N; i += kPickThreads) {
            p.out_commit[out + i] = -1;
            tp.out_path[out + i] = -1;
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
    for (int i = tid; i < n; i += kPickThreads) {
        const int up = i ? tp.parent[out + i] : -1;
        tree.token[i] = p.block[out + i];
        tree.parent[i] = up < i ? up : -1;               // (a parent comes before its children)
        tree.next[i] = -1;
    }
    for (int i = warp; i < n; i += kPickThreads / 32) {
        const Stat v = row_stat(p, b, i, inv_t, lane);
        if (lane == 0) tree.row[i] = v;
    }
    __syncthreads();
    // each node against its parent's row
    for (int i = tid; i < n; i += kPickThreads) {
        const int up = tree.parent[i], t = tree.token[i];
        float w = 0.0f;
        if (up >= 0 && t >= 0 && t < p.V) {
            const Stat &v = tree.row[up];
            if (greedy) w = v.m > -INFINITY && t == v.at ? 1.0f : 0.0f;
            else if (v.m > -INFINITY) w = weight(logit(rows + up * p.lp, t), v.m, inv_t) / v.s;
            for (int j = up + 1; j < i; ++j)
                if (tree.parent[j] == up && tree.token[j] == t) w = 0.0f;
        }
        tree.weight[i] = w;
    }
    __syncthreads();
    for (int i = tid; i < n; i += kPickThreads) {
        const int up = tree.parent[i];
        if (up < 0) continue;
        float before = 0.0f;
        for (int j = up + 1; j < i; ++j)
            if (tree.parent[j] == up) before += tree.weight[j];
        const float u = greedy ? 0.0f : p.u[out + up];
        if (u < before + tree.weight[i] && !(u < before)) tree.next[up] = i;
    }
    __syncthreads();
    if (tid == 0) {
        int a = 0, at = 0;
        tree.path[0] = 0;
        while (tree.next[at] >= 0) tree.path[++a] = at = tree.next[at];
        tree.accepted = a;
        tree.kid_count = 0;
    }
    __syncthreads();
    const int a = tree.accepted, end = tree.path[a];
    const Stat row = tree.row[end];
    const T *x = rows + end * p.lp;
    int32_t token = row.m > -INFINITY ? row.at : -1;
    if (!greedy) {
        cluster_arrive();                                // every CTA runs before another writes to it
        for (int i = end + 1 + tid; i < n; i += kPickThreads)
            if (tree.parent[i] == end) tree.kids[atomicAdd(&tree.kid_count, 1)] = tree.token[i];
        __syncthreads();
        const int kids = tree.kid_count;
        auto proposed = [&](int j) {
            for (int k = 0; k < kids; ++k)
                if (tree.kids[k] == j) return true;
            return false;
        };
        const float *noise = p.noise + int64_t(b) * p.V;
        const float c = inv_t * 1.4426950408889634f;
        Best best{0.0f, INT32_MAX};
        // keys without the common factor 1 / s.  The best of kRace keys first; which one it was
        // only where it beats the thread's best.
        if (row.m > -INFINITY && row.m <= FLT_MAX && c <= FLT_MAX)
            for (int j0 = lo + tid; j0 < hi; j0 += kRace * kPickThreads) {
                float key[kRace], es[kRace];
#pragma unroll
                for (int k = 0; k < kRace; ++k) {
                    const int j = min(j0 + k * kPickThreads, hi - 1);        // past the end: the last one again
                    key[k] = to_f32(x[j]);
                    es[k] = __ldcs(noise + j);
                }
                float top = 0.0f;                        // NaN drops out
#pragma unroll
                for (int k = 0; k < kRace; ++k) {
                    key[k] = __fdividef(exp2_approx((key[k] - row.m) * c), es[k]);
                    top = fmaxf(top, key[k]);
                }
                if (top > best.key) {
#pragma unroll
                    for (int k = 0; k < kRace; ++k) {
                        const int j = min(j0 + k * kPickThreads, hi - 1);
                        if (key[k] > best.key && !proposed(j)) best = Best{key[k], j};
                    }
                }
            }
        __syncwarp();                                    // the cluster's barrier wants whole warps
        cluster_wait();
        best = cluster_best(best, warps[0], places[0], rank, p.cluster);
        if (best.key == 0.0f && row.m > -INFINITY) {
            // nothing left above 2^-126, or infinite logits: once more, to the smallest
            // float32, with p's own best should there be nothing at all without the children's
            Best all{0.0f, INT32_MAX};
            for (int j = lo + tid; j < hi; j += kPickThreads) {
                const float own = weight(logit(x, j), row.m, inv_t) / noise[j];
                if (own > best.key && !proposed(j)) best = Best{own, j};
                if (own > all.key) all = Best{own, j};
            }
            best = cluster_best(best, warps[1], places[1], rank, p.cluster);
            all = cluster_best(all, warps[2], places[2], rank, p.cluster);
            if (best.key == 0.0f) best = all;
        }
        if (rank) return;
        token = best.key > 0.0f ? best.at : -1;
    }
    for (int k = tid; k < N; k += kPickThreads) {
        const int node = k < a ? tree.path[k + 1] : -1;
        const int32_t t = k < a ? tree.token[node] : k == a ? token : -1;
        p.out_commit[out + k] = t;
        tp.out_path[out + k] = node;
        if (!lps) continue;
        float v = 0.0f;
        if (t >= 0) {
            const int from = tree.path[k];
            const Stat &s = tree.row[from];
            const float z = logit(rows + from * p.lp, t);
            v = (z == s.m ? 0.0f : (z - s.m) * inv_t) - logf(s.s);
        }
        lps[k] = v;
    }
    if (tid == 0) {
        p.out_accepted[b] = a;
        p.out_ncommit[b] = a + (token >= 0);
    }
}

template <typename T>
int launch(const TreeParams &tp, cudaStream_t stream) {
    const int rc = launch_stats<T>(tp.rows, stream);
    return rc != LOOKUP_DRAFT_OK ? rc
                                 : launch_clusters(walk_kernel<T>, tp.rows.B, tp.rows.cluster, kPickThreads, 0, stream, tp);
}

}  // namespace

extern "C" {

size_t lookup_verify_tree_workspace_bytes(int32_t B, int32_t N, int32_t V) {
    if (B < 0 || N < 1 || N > LOOKUP_TREE_MAX_NODES || V < 1 || V >= kMaxV) return 0;
    return size_t(B) * size_t(N) * size_t(std::max(segments(B, N - 1, V, 4), segments(B, N - 1, V, 2))) * sizeof(float4) +
           kMaxCtas * sizeof(int32_t);
}

int lookup_verify_tree(const int32_t *tokens, const int32_t *parent, const int32_t *n, const void *logits,
                       const int64_t *logits_strides, int32_t type, int32_t V, const float *noise,
                       const float *temperature, const float *u, int32_t B, int32_t N, int32_t *out_accepted,
                       int32_t *out_commit, int32_t *out_ncommit, int32_t *out_path, float *out_logprobs,
                       void *workspace, size_t workspace_bytes, struct CUstream_st *stream) {
    lkd::TraceRange trace_("lookup_verify_tree");
    if (B < 0 || N < 1 || N > LOOKUP_TREE_MAX_NODES || V < 1 || V >= kMaxV) return LOOKUP_DRAFT_EINVAL;
    if (type != LOOKUP_TYPE_F32 && type != LOOKUP_TYPE_F16 && type != LOOKUP_TYPE_BF16) return LOOKUP_DRAFT_EINVAL;
    if (B == 0) return LOOKUP_DRAFT_OK;
    const int64_t segs = segments(B, N - 1, V, type == LOOKUP_TYPE_F32 ? 4 : 2);
    if (segs > INT32_MAX / (int64_t(B) * N) || int64_t(B) * kMaxCluster > INT32_MAX) return LOOKUP_DRAFT_EINVAL;
    if (!tokens || !parent || !n || !logits || !logits_strides || !out_accepted || !out_commit || !out_ncommit ||
        !out_path || !workspace || (noise && N > 1 && !u))
        return LOOKUP_DRAFT_EINVAL;
    if (misaligned(logits, type == LOOKUP_TYPE_F32 ? 4 : 2) || misaligned(workspace, 16)) return LOOKUP_DRAFT_EINVAL;
    for (const void *q : {static_cast<const void *>(tokens), static_cast<const void *>(parent), static_cast<const void *>(n),
                          static_cast<const void *>(noise), static_cast<const void *>(temperature),
                          static_cast<const void *>(u), static_cast<const void *>(out_accepted),
                          static_cast<const void *>(out_commit), static_cast<const void *>(out_ncommit),
                          static_cast<const void *>(out_path), static_cast<const void *>(out_logprobs)})
        if (misaligned(q, 4)) return LOOKUP_DRAFT_EINVAL;
    if (workspace_bytes < lookup_verify_tree_workspace_bytes(B, N, V)) return LOOKUP_DRAFT_EINVAL;
    int sms = 0;
    const int rc = lkd::sm_count(&sms);
    if (rc != LOOKUP_DRAFT_OK) return rc;
    TreeParams tp{};
    Params &p = tp.rows;
    p.block = tokens, p.len = n, p.logits = logits, p.lb = logits_strides[0], p.lp = logits_strides[1], p.root = 1;
    p.noise = noise, p.temperature = noise ? temperature : nullptr, p.u = u;
    p.B = B, p.P = N - 1, p.V = V, p.segs = int32_t(segs), p.cluster = cluster_for(B, V);
    p.out_accepted = out_accepted, p.out_commit = out_commit, p.out_ncommit = out_ncommit, p.out_logprobs = out_logprobs;
    tp.parent = parent, tp.out_path = out_path;
    const int64_t units = int64_t(B) * N * segs;
    p.ctas = int32_t(std::min<int64_t>(units, std::min(sms, kMaxCtas)));
    p.part = static_cast<float4 *>(workspace);
    p.status = reinterpret_cast<int32_t *>(p.part + units);
    p.limit = 2 * lookup_wait_limit_ns();                // at 2 GHz
    if (type == LOOKUP_TYPE_F32) return launch<float>(tp, stream);
    if (type == LOOKUP_TYPE_F16) return launch<__half>(tp, stream);
    return launch<__nv_bfloat16>(tp, stream);
}

}  // extern "C"
