// ssd_tree.cu -- a tree of drafted tokens: masks and positions from its parents, and the walk of
// the target's draws down it (sm_103a).
//
// Both hold a sequence's parents in shared memory, have a thread for each node and are bound by
// latency: a batch of 256 trees of 37 nodes is 40 KB, and one of 48 trees of up to 509 nodes writes
// 0.8 MB of masks.  The first takes 7.3 us either way, a launch with cold caches and little else.
#include "ssd_kv.h"

namespace ssd {
namespace {

constexpr int kTreeThreads = 128;

struct TreeSeq {
    int first, n;  // first token, nodes served
    int to;        // end of its tokens
    bool fits;
};
__device__ __forceinline__ TreeSeq tree_seq(const int32_t *cu, int b, int T, int max_new) {
    const int first = cu[b], next = cu[b + 1];
    TreeSeq s;
    s.first = min(max(first, 0), T);
    s.to = min(max(next, s.first), T);
    s.n = min(s.to - s.first, max_new);
    s.fits = first >= 0 && next >= first && next <= T && s.to - s.first <= max_new;
    return s;
}

struct TreePlanParams {
    const int32_t *parent, *cu, *seq_len;
    int B, T, max_new, words;
    int32_t *positions, *mask;
    int32_t *dev_status;
};

// A thread walks from its node to the root.  Parents lie before their children, so the words of the
// mask are finished from the last one down and none is kept.  A CTA takes kTreeThreads nodes of a
// sequence and needs the parents up to its last one: a row's words are written one by one, 32 rows
// to an instruction, which four SMs do faster than one (48 trees of up to 509 nodes, 11.4 and 16.5
// us).  Every CTA looks through all token counts for a fall: of 4096 sequences that takes 4 us of 20,
// of 1024 none that can be seen.
__global__ void __launch_bounds__(kTreeThreads) tree_plan_kernel(const __grid_constant__ TreePlanParams P) {
    __shared__ int32_t up[SSD_TREE_MAX];
    __shared__ int room;
    const int b = blockIdx.x;
    TreeSeq s = tree_seq(P.cu, b, P.T, P.max_new);
    int bad = s.fits ? 0 : SSD_DEV_BAD_LENGTH;
    const int seqs = sequences<kTreeThreads>(P.cu, P.B, &room);
    if (b >= seqs) s.n = 0, s.to = s.first;
    int base = P.seq_len[b];
    if (base < 0 || base > 0x7FFFFFFF - SSD_TREE_MAX) base = 0, bad |= SSD_DEV_BAD_LENGTH;
    const int from = static_cast<int>(blockIdx.y) * kTreeThreads;
    for (int i = threadIdx.x; i < min(s.n, from + kTreeThreads); i += kTreeThreads) {
        int p = P.parent[s.first + i];
        if (p < -1 || p >= i) p = -1, bad |= SSD_DEV_BAD_TREE;
        up[i] = p;
    }
    __syncthreads();
    for (int i = from + static_cast<int>(threadIdx.x); i < s.to - s.first; i += static_cast<int>(gridDim.y) * kTreeThreads) {
        const int64_t t = s.first + i;
        int32_t *mask = P.mask + t * P.words;
        int w = P.words, depth = -1;
        uint32_t bits = 0;
        for (int a = i < s.n ? i : -1; a >= 0; a = up[a], ++depth) {
            const int at = a >> 5;
            if (at != w) {
                if (w < P.words) mask[w] = static_cast<int32_t>(bits);
                while (--w > at) mask[w] = 0;
                bits = 0;
            }
            bits |= 1u << (a & 31);
        }
        if (w < P.words) mask[w] = static_cast<int32_t>(bits);
        while (--w >= 0) mask[w] = 0;
        P.positions[t] = depth < 0 ? 0 : base + depth;
    }
    // entries behind the last sequence
    const int end = min(max(P.cu[seqs], 0), P.T), block = static_cast<int>(blockIdx.y * gridDim.x) + b;
    const int64_t stride = static_cast<int64_t>(gridDim.x) * gridDim.y * kTreeThreads;
    for (int64_t t = static_cast<int64_t>(end) + static_cast<int64_t>(block) * kTreeThreads + threadIdx.x; t < P.T; t += stride) {
        P.positions[t] = 0;
        for (int w = 0; w < P.words; ++w) P.mask[t * P.words + w] = 0;
    }
    report(P.dev_status, bad);
}

struct TreeAcceptParams {
    const int32_t *parent, *tokens, *sampled, *cu;
    int B, T, max_new, max_path;
    int32_t *accept_len, *bonus, *path;
    int32_t *dev_status;
};

// Every node looks whether its token is its parent's draw; the first such child is where the walk
// goes on.  What is left for one thread is a chain of reads from shared memory.  The block has a
// thread for each node, so that what it reads is on its way at once (trees of up to 509 nodes, 8.3
// us, 13.4 with 128 threads).
__global__ void __launch_bounds__(SSD_TREE_MAX) tree_accept_kernel(const __grid_constant__ TreeAcceptParams P) {
    __shared__ int32_t draw[SSD_TREE_MAX], next[SSD_TREE_MAX];
    __shared__ int32_t walk[SSD_MAX_K + 1];
    const int b = blockIdx.x;
    const TreeSeq s = tree_seq(P.cu, b, P.T, P.max_new);
    int bad = s.fits ? 0 : SSD_DEV_BAD_LENGTH;
    const int i = static_cast<int>(threadIdx.x);
    int parent = -1, token = 0;
    if (i < s.n) {
        parent = P.parent[s.first + i], token = P.tokens[s.first + i];
        draw[i] = P.sampled[s.first + i];
        next[i] = 0x7FFFFFFF;
    }
    if (i < P.max_path) walk[i] = -1;
    __syncthreads();
    if (parent < -1 || parent >= i)
        bad |= SSD_DEV_BAD_TREE;
    else if (parent >= 0 && token == draw[parent])
        atomicMin(&next[parent], i);
    __syncthreads();
    if (i == 0) {
        int length = 0, last = -1;
        for (int node = s.n > 0 ? 0 : 0x7FFFFFFF; node < s.n && length < P.max_path; node = next[node]) {
            walk[length++] = node;
            last = draw[node];
            if (last < 0) break;
        }
        if (length > 0 && last < 0) {
            bad |= SSD_DEV_BAD_TOKEN;
            while (length > 0) walk[--length] = -1;
        }
        P.accept_len[b] = length - 1;
        P.bonus[b] = last < 0 ? -1 : last;
    }
    __syncthreads();
    if (i < P.max_path) P.path[static_cast<int64_t>(b) * P.max_path + i] = walk[i];
    report(P.dev_status, bad);
}
constexpr int kAcceptLeast = 64;  // threads: one for each place of a path, too
static_assert(SSD_MAX_K + 1 <= kAcceptLeast, "");

}  // namespace
}  // namespace ssd

extern "C" int ssd_tree_plan(const int32_t *parent, const int32_t *cu_new, const int32_t *seq_len, int B, int T,
                             int max_new, int32_t *positions, int32_t *mask, int32_t *dev_status, void *stream) {
    using namespace ssd;
    if (!cu_new || !seq_len || (T > 0 && (!parent || !positions || !mask))) return SSD_ERR_INVALID_ARG;
    if (B < 1 || T < 0 || max_new < 1) return SSD_ERR_INVALID_ARG;
    if (B > SSD_KV_MAX_B || max_new > SSD_TREE_MAX) return SSD_ERR_UNSUPPORTED;
    if (T == 0) return SSD_OK;
    const TreePlanParams P{parent, cu_new, seq_len, B, T, max_new, (max_new + 31) / 32, positions, mask, dev_status};
    const dim3 grid(static_cast<unsigned>(B), static_cast<unsigned>((max_new + kTreeThreads - 1) / kTreeThreads));
    tree_plan_kernel<<<grid, kTreeThreads, 0, static_cast<cudaStream_t>(stream)>>>(P);
    return launched();
}

extern "C" int ssd_tree_accept(const int32_t *parent, const int32_t *tokens, const int32_t *sampled,
                               const int32_t *cu_new, int B, int T, int max_new, int max_path, int32_t *accept_len,
                               int32_t *bonus, int32_t *path, int32_t *dev_status, void *stream) {
    using namespace ssd;
    if (!cu_new || !accept_len || !bonus || !path || (T > 0 && (!parent || !tokens || !sampled))) return SSD_ERR_INVALID_ARG;
    if (B < 1 || T < 0 || max_new < 1 || max_path < 1 || max_path > SSD_MAX_K + 1) return SSD_ERR_INVALID_ARG;
    if (B > SSD_KV_MAX_B || max_new > SSD_TREE_MAX) return SSD_ERR_UNSUPPORTED;
    const TreeAcceptParams P{parent, tokens, sampled, cu_new, B, T, max_new, max_path, accept_len, bonus, path, dev_status};
    const int threads = max_new > kAcceptLeast ? (max_new + 31) / 32 * 32 : kAcceptLeast;
    tree_accept_kernel<<<static_cast<unsigned>(B), threads, 0, static_cast<cudaStream_t>(stream)>>>(P);
    return launched();
}
