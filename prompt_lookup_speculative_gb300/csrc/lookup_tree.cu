// lookup_tree.cu -- chains of proposals merged into a tree, and the accepted branch's
// cache rows moved to the front of the block.
//
// The contracts are in include/lookup_tree.h (lookup_tree_merge, lookup_kv_compact).
//
// Merging.  Entered one after another, position j of chain c becomes a new node exactly
// where no earlier chain begins with the same j + 1 tokens.  With l(c, c') the number of
// tokens that two chains begin with alike and s(c) = max over c' < c of l(c, c'), chain c
// makes the nodes of its positions s(c) .. len(c) - 1, numbered from 1 + the sum of
// len - s over the chains before; position j < s(c) is the node of the earliest chain c'
// with l(c, c') > j, which made it.  So nothing is sequential: all l, then a sum over the
// chains, then every position's node, then its ancestors.  Numbers from N on are left
// out, and with them all that would hang on them, whose numbers are larger.
// What bounds it: a warp's own instructions, 2700 for 16 chains of 8 (all pairs compared, every
// position's first chain looked for, every node's ancestors gathered from its chain's start),
// each waiting for the one before: the issue slots are 61% busy.  4096 such requests: 23.2 us, and
// a copy of their bytes takes 1.1; one with 2 chains of 7: 3.4 us, 8.9 as called.

#include "lookup_draft.h"
#include "lookup_tree.h"
#include "common.cuh"

#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>
#include <vector>

namespace {

using lkd::allow_dependent_launch;
using lkd::launch_pdl;
using lkd::wait_for_prerequisite_grid;

bool misaligned(const void *p, size_t to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) != 0; }

// ------------------------------------------------------------------- merging ----
constexpr int kMaxChains = 64, kMaxPositions = 4096;
constexpr int kMergeWarps = 4;           // requests of a CTA where their chains fit 48 KB of shared memory

struct MergeParams {
    const int32_t *root, *chains, *len;
    int32_t B, C, K, N, words, warps;
    int32_t *tokens, *parent, *depth;
    int64_t *mask;
    int32_t *n;
};

// Shared memory of a request: its chains' tokens, rows of an odd number of words (lanes
// that look at one position of different chains use different banks), the nodes of their
// positions, l of all pairs, and per chain its length, s and first number.
struct MergeSmem {
    int32_t row, tokens, nodes, alike, lens, starts, bases, bytes;
    __host__ __device__ MergeSmem(int C, int K) {
        row = K | 1;
        tokens = 0;
        lens = tokens + C * row * 4;
        starts = lens + C * 4;
        bases = starts + C * 4;
        nodes = bases + C * 4;
        alike = nodes + (C * K * 2 + 3) / 4 * 4;
        bytes = alike + (C * C * 2 + 15) / 16 * 16;
        bytes = (bytes + 15) / 16 * 16;
    }
};

__global__ void __launch_bounds__(32 * kMergeWarps) merge_kernel(const __grid_constant__ MergeParams p) {
    extern __shared__ __align__(16) unsigned char smem[];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t b = int64_t(blockIdx.x) * p.warps + warp;
    wait_for_prerequisite_grid();
    allow_dependent_launch();
    if (b >= p.B) return;
    const int C = p.C, K = p.K, N = p.N;
    const MergeSmem at(C, K);
    unsigned char *mine = smem + warp * at.bytes;
    int32_t *tok = reinterpret_cast<int32_t *>(mine + at.tokens), *lens = reinterpret_cast<int32_t *>(mine + at.lens);
    int32_t *starts = reinterpret_cast<int32_t *>(mine + at.starts), *bases = reinterpret_cast<int32_t *>(mine + at.bases);
    uint16_t *nodes = reinterpret_cast<uint16_t *>(mine + at.nodes), *alike = reinterpret_cast<uint16_t *>(mine + at.alike);
    const int32_t *chains = p.chains + b * C * K;
    for (int x = lane; x < C * K; x += 32) tok[x / K * at.row + x % K] = chains[x];
    for (int c = lane; c < C; c += 32) lens[c] = min(max(p.len[b * C + c], 0), K);
    __syncwarp();
    for (int c = lane; c < C; c += 32) {                 // up to the first negative token
        int n = 0;
        while (n < lens[c] && tok[c * at.row + n] >= 0) ++n;
        lens[c] = n;
    }
    __syncwarp();
    for (int x = lane; x < C * C; x += 32) {             // l of each chain and those before it
        const int c = x / C, d = x % C;
        if (d >= c) continue;
        const int most = min(lens[c], lens[d]);
        int n = 0;
        while (n < most && tok[c * at.row + n] == tok[d * at.row + n]) ++n;
        alike[x] = uint16_t(n);
    }
    __syncwarp();
    int before = 1;                                      // nodes of the chains ahead of these 32
    for (int c0 = 0; c0 < C; c0 += 32) {
        const int c = c0 + lane;
        int s = 0, made = 0;
        if (c < C) {
            for (int d = 0; d < c; ++d) s = max(s, int(alike[c * C + d]));
            made = lens[c] - s;
        }
        int upto = made;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, upto, d);
            if (lane >= d) upto += y;
        }
        if (c < C) {
            starts[c] = s;
            bases[c] = before + upto - made;
        }
        before += __shfl_sync(0xffffffffu, upto, 31);
    }
    const int n = min(before, N);
    __syncwarp();
    for (int x = lane; x < C * K; x += 32) {             // every position's node
        const int c = x / K, j = x % K;
        if (j >= lens[c]) continue;
        int d = 0;
        while (d < c && alike[c * C + d] <= j) ++d;      // the first chain with this beginning
        nodes[x] = uint16_t(min(bases[d] + j - starts[d], N));
    }
    __syncwarp();
    int32_t *tokens = p.tokens + b * N, *parent = p.parent + b * N, *depth = p.depth + b * N;
    int64_t *mask = p.mask + b * N * p.words;
    for (int x = lane; x < C * K; x += 32) {             // what the new ones are
        const int c = x / K, j = x % K;
        if (j < starts[c] || j >= lens[c]) continue;
        const int node = nodes[x];
        if (node >= N) continue;
        tokens[node] = tok[c * at.row + j];
        parent[node] = j ? nodes[x - 1] : 0;
        depth[node] = j + 1;
        for (int w = 0; w < p.words; ++w) {
            uint64_t bits = w ? 0 : 1;
            for (int k = 0; k <= j; ++k) {
                const int a = nodes[x - j + k];
                if (a / 64 == w) bits |= uint64_t(1) << (a % 64);
            }
            mask[node * p.words + w] = int64_t(bits);
        }
    }
    for (int i = lane; i < N; i += 32)
        if (i == 0 || i >= n) {
            tokens[i] = i ? -1 : p.root[b];
            parent[i] = -1;
            depth[i] = 0;
            for (int w = 0; w < p.words; ++w) mask[i * p.words + w] = i == 0 && w == 0;
        }
    if (lane == 0) p.n[b] = n;
}

// ---------------------------------------------------------------- compaction ----
// Row by row, the accepted branch moves down: position path[j] >= j + 1 to j + 1.  A place
// that is written may be the source of an earlier move, never of a later one, since both
// sides rise; so a thread that takes the moves in their order for its own 16 bytes of
// every row needs no copy and no barrier.
// What bounds it: the moved rows' bytes, read and written once; all layers in one launch.
// 64 requests, 32 layers with 8 heads of 128: 16.9 us for 71 MB (4.2 TB/s); 74 to 82 as called,
// most of it what the caller takes to list 64 tensors.  30 moves each, all by one row: 85 us for
// 503 MB (5.9 TB/s).  Four layers of one request: 2.4 us, 21 to 23 as called.
constexpr int kMoveThreads = 256;
constexpr int kMoveBatch = 8;            // moves in flight per thread
constexpr int kMoveLayers = 128;         // of a launch

struct CompactParams {
    void *caches[2 * kMoveLayers];       // k and v of each layer, k first
    const int32_t *table, *kv_len, *path, *accepted;
    int32_t *status;
    int32_t B, N, Hkv, D, max_pages, pages, page_shift, caches_n, slices;
};

template <typename U>
__global__ void __launch_bounds__(kMoveThreads) compact_kernel(const __grid_constant__ CompactParams p) {
    __shared__ int64_t from[LOOKUP_TREE_MAX_NODES], to[LOOKUP_TREE_MAX_NODES];
    __shared__ int s_moves;
    const int tid = threadIdx.x, lane = tid & 31;
    const int b = blockIdx.x / p.slices, slice = blockIdx.x % p.slices;
    wait_for_prerequisite_grid();
    allow_dependent_launch();
    const int a = p.accepted[b];
    if (tid < 32) {                                      // the moves: rows of kv head 0
        const int64_t kv = max(p.kv_len[b], 0);
        const int32_t *path = p.path + int64_t(b) * p.N;
        auto slot = [&](int64_t pos) -> int64_t {
            const int64_t at = pos >> p.page_shift;
            const int32_t page = at < p.max_pages ? p.table[int64_t(b) * p.max_pages + at] : -1;
            if (page < 0 || page >= p.pages) return -1;
            return ((int64_t(page) * p.Hkv) << p.page_shift) + (pos & ((int64_t(1) << p.page_shift) - 1));
        };
        bool bad = a > p.N;
        int moves = 0;
        for (int j0 = 0; j0 < min(a, p.N); j0 += 32) {
            const int j = j0 + lane;
            bool move = false;
            int64_t src = 0, dst = 0;
            if (j < min(a, p.N)) {
                const int node = path[j], last = j ? path[j - 1] : 0;
                if (node <= last || node >= LOOKUP_TREE_MAX_NODES) {
                    bad = true;
                } else {
                    src = slot(kv + node);
                    dst = slot(kv + 1 + j);
                    bad = bad || src < 0 || dst < 0;
                    move = node != j + 1;
                }
            }
            const unsigned all = __ballot_sync(0xffffffffu, move);
            if (move) {
                const int k = moves + __popc(all & ((1u << lane) - 1));
                from[k] = src;
                to[k] = dst;
            }
            moves += __popc(all);
        }
        bad = __any_sync(0xffffffffu, bad);
        if (lane == 0) {
            s_moves = bad ? 0 : moves;
            if (p.status && slice == 0) p.status[b] = bad ? 1 : 0;
        }
    }
    __syncthreads();
    const int moves = s_moves;
    if (moves == 0) return;
    const int per = p.D * 2 / int(sizeof(U));            // pieces of a row
    const int units = p.caches_n * p.Hkv * per;
    for (int x = slice * kMoveThreads + tid; x < units; x += p.slices * kMoveThreads) {
        const int piece = x % per, rest = x / per;
        const int h = rest % p.Hkv, cache = rest / p.Hkv;
        U *base = static_cast<U *>(p.caches[cache]) + (int64_t(h) << p.page_shift) * per + piece;
        for (int k0 = 0; k0 < moves; k0 += kMoveBatch) {
            U v[kMoveBatch];
#pragma unroll
            for (int k = 0; k < kMoveBatch; ++k)
                if (k0 + k < moves) v[k] = base[from[k0 + k] * per];
#pragma unroll
            for (int k = 0; k < kMoveBatch; ++k)
                if (k0 + k < moves) base[to[k0 + k] * per] = v[k];
        }
    }
}

}  // namespace

extern "C" {

int lookup_tree_merge(const int32_t *root, const int32_t *chains, const int32_t *len, int32_t B, int32_t C, int32_t K,
                      int32_t N, int32_t *tokens, int32_t *parent, int32_t *depth, int64_t *mask, int32_t *n,
                      struct CUstream_st *stream) {
    lkd::TraceRange trace_("lookup_tree_merge");
    if (B < 0 || C < 0 || K < 0 || C > kMaxChains || int64_t(C) * K > kMaxPositions || N < 1 || N > LOOKUP_TREE_MAX_NODES)
        return LOOKUP_DRAFT_EINVAL;
    if (B == 0) return LOOKUP_DRAFT_OK;
    if (C * K == 0) C = K = 0;
    if (!root || (C && (!chains || !len)) || !tokens || !parent || !depth || !mask || !n) return LOOKUP_DRAFT_EINVAL;
    for (const void *x : {static_cast<const void *>(root), static_cast<const void *>(chains), static_cast<const void *>(len),
                          static_cast<const void *>(tokens), static_cast<const void *>(parent),
                          static_cast<const void *>(depth), static_cast<const void *>(n)})
        if (misaligned(x, 4)) return LOOKUP_DRAFT_EINVAL;
    if (misaligned(mask, 8)) return LOOKUP_DRAFT_EINVAL;
    MergeParams p{root, chains, len, B, C, K, N, (N + 63) / 64, kMergeWarps, tokens, parent, depth, mask, n};
    const MergeSmem each(C, K);
    if (each.bytes * p.warps > 48 * 1024) p.warps = 1;
    static_assert((kMaxPositions + kMaxChains) * 4 + kMaxPositions * 2 + 3 * kMaxChains * 4 +
                      kMaxChains * kMaxChains * 2 + 64 <= 48 * 1024,
                  "a request's chains fit the shared memory that needs no opt-in");
    return launch_pdl(merge_kernel, unsigned((int64_t(B) + p.warps - 1) / p.warps), unsigned(32 * p.warps), stream, p,
                      size_t(each.bytes) * p.warps);
}

int lookup_kv_compact(void *const *k_caches, void *const *v_caches, int32_t layers, const int32_t *block_table,
                      const int32_t *kv_len, const int32_t *path, const int32_t *accepted, int32_t B, int32_t N,
                      int32_t Hkv, int32_t D, int32_t max_pages, int32_t pages, int32_t page_size, int32_t *status,
                      struct CUstream_st *stream) {
    lkd::TraceRange trace_("lookup_kv_compact");
    if (layers < 0 || B < 0 || N < 0 || N > LOOKUP_TREE_MAX_NODES || Hkv < 1 || D < 1 || D > 1024 || max_pages < 1 ||
        pages < 1 || page_size < 1 || (page_size & (page_size - 1)))
        return LOOKUP_DRAFT_EINVAL;
    if (int64_t(Hkv) * D > INT32_MAX / (4 * kMoveLayers)) return LOOKUP_DRAFT_EINVAL;
    if (B == 0) return LOOKUP_DRAFT_OK;
    if ((layers && (!k_caches || !v_caches)) || !block_table || !kv_len || (N && !path) || !accepted)
        return LOOKUP_DRAFT_EINVAL;
    for (const void *x : {static_cast<const void *>(block_table), static_cast<const void *>(kv_len),
                          static_cast<const void *>(path), static_cast<const void *>(accepted),
                          static_cast<const void *>(status)})
        if (misaligned(x, 4)) return LOOKUP_DRAFT_EINVAL;
    bool wide = D % 8 == 0;
    // no two of the caches share memory: their moves would be made twice, in no order
    std::vector<uintptr_t> starts;
    try {
        starts.reserve(2 * size_t(layers));
    } catch (...) {
        return lookup_record_cuda_error(cudaErrorMemoryAllocation, "host memory");
    }
    for (int32_t l = 0; l < layers; ++l)
        for (void *x : {k_caches[l], v_caches[l]}) {
            if (!x || misaligned(x, 2)) return LOOKUP_DRAFT_EINVAL;
            wide = wide && !misaligned(x, 16);
            starts.push_back(reinterpret_cast<uintptr_t>(x));
        }
    std::sort(starts.begin(), starts.end());
    const uint64_t bytes = uint64_t(pages) * uint64_t(Hkv) * uint64_t(page_size) * uint64_t(D) * 2;
    for (size_t k = 1; k < starts.size(); ++k)
        if (starts[k] - starts[k - 1] < bytes) return LOOKUP_DRAFT_EINVAL;
    int sms = 0;
    const int rc = lkd::sm_count(&sms);
    if (rc != LOOKUP_DRAFT_OK) return rc;
    CompactParams p{};
    p.table = block_table, p.kv_len = kv_len, p.path = path, p.accepted = accepted;
    p.B = B, p.N = N, p.Hkv = Hkv, p.D = D, p.max_pages = max_pages, p.pages = pages;
    while ((1 << p.page_shift) < page_size) ++p.page_shift;
    int32_t l = 0;
    do {                                                 // (no layers: the status alone)
        const int32_t some = std::min(layers - l, kMoveLayers);
        for (int32_t k = 0; k < some; ++k) {
            p.caches[2 * k] = k_caches[l + k];
            p.caches[2 * k + 1] = v_caches[l + k];
        }
        p.caches_n = 2 * some;
        p.status = l == 0 ? status : nullptr;
        const int64_t units = int64_t(p.caches_n) * Hkv * (wide ? D / 8 : D);
        // CTAs of a request: a unit per thread, while the grid stays within eight CTAs per SM
        const int64_t most = std::max<int64_t>(int64_t(8) * sms / B, 1);
        p.slices = int32_t(std::max<int64_t>(std::min((units + kMoveThreads - 1) / kMoveThreads, most), 1));
        if (int64_t(B) * p.slices > INT32_MAX) return LOOKUP_DRAFT_EINVAL;
        const int got = launch_pdl(wide ? compact_kernel<uint4> : compact_kernel<uint16_t>, unsigned(B * p.slices),
                                   unsigned(kMoveThreads), stream, p);
        if (got != LOOKUP_DRAFT_OK) return got;
        l += some;
    } while (l < layers);
    return LOOKUP_DRAFT_OK;
}

}  // extern "C"
