// ssd_kv_plan.cu -- block tables and slot maps from request lengths, on the GPU
// (sm_103a).
//
// [SSD] "Speculative Speculative Decoding" notes (papernotes.org), "整体框架": after a
// round the KV pages of each sequence are reconciled with what was accepted.  Here one
// launch commits the accepted lengths, gives back the pages beyond them, takes pages for
// the tokens that come next, and writes their slots and positions.
//
// Three prefix sums over the batch decide everything: of the new tokens (their places in
// the packed token order), of the pages taken and of the pages given back (their places
// in the ring).  What follows is one independent write per page or token, found by binary
// search in those sums.  The bytes are few (a batch of 256 moves 20 KB), so latency
// bounds the call: one launch, every CTA of one cluster computing the same sums from
// shared memory instead of waiting for one that does.  Captured into a graph, 256 requests
// of 5 tokens take 13 us and 48 of up to 2700 tokens 21, of which an empty launch is 7.
#include <cooperative_groups.h>

#include <atomic>

#include "ssd_kv.h"

namespace ssd {
namespace {

namespace cg = cooperative_groups;

constexpr int kPlanThreads = 512;
constexpr int kPlanWarps = kPlanThreads / 32;
constexpr int kSumsBytes = 6 * sizeof(int32_t);  // of shared memory for each request
constexpr int kPlanCtas = 8;                     // at most, of one cluster
constexpr int kTokens = 4;                       // that a thread looks up at once
// the tokens of one turn of the whole cluster: a token's index stays in 32 bits for caps that leave room for one
constexpr int kTurn = kPlanCtas * kPlanThreads * kTokens;

struct PlanParams {
    int32_t *seq_len;
    const int32_t *accept_len;
    const int32_t *new_len;
    int32_t *held;
    int B;
    int32_t *block_table;
    int max_blocks;
    int32_t *ring;
    int32_t *ring_state;
    int num_pages;
    int page_shift;
    int cap;
    int32_t *cu_new;
    int32_t *kv_len;
    int32_t *slots;
    int32_t *positions;
    int32_t *dev_status;
};

// Inclusive prefix sum over the block of one 64-bit value per thread, added to `carry`
// (the total is added to carry for the next call).
__device__ __forceinline__ uint64_t block_scan(uint64_t v, uint64_t &carry, uint64_t *red) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint64_t t = __shfl_up_sync(0xFFFFFFFFu, v, o);
        if (lane >= o) v += t;
    }
    __syncthreads();
    if (lane == 31) red[warp] = v;
    __syncthreads();
    uint64_t before = 0, total = 0;
#pragma unroll
    for (int w = 0; w < kPlanWarps; ++w) {
        const uint64_t t = red[w];
        if (w < warp) before += t;
        total += t;
    }
    const uint64_t r = carry + before + v;
    carry += total;
    return r;
}

// First index b in [0, n) with sums[b] > x (sums ascending, sums[n-1] > x).
__device__ __forceinline__ int first_above(const int32_t *sums, int n, int x) {
    int lo = 0, hi = n - 1;
    while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (sums[mid] > x)
            hi = mid;
        else
            lo = mid + 1;
    }
    return lo;
}

__global__ void __launch_bounds__(kPlanThreads) plan_kernel(const __grid_constant__ PlanParams P) {
    extern __shared__ int32_t sums[];  // 6 arrays of B
    __shared__ uint64_t red[kPlanWarps];
    __shared__ int granted_sh;
    const int B = P.B;
    int32_t *cu = sums;           // inclusive sums of the new tokens
    int32_t *take = cu + B;       // inclusive sums of the pages taken
    int32_t *give = take + B;     // inclusive sums of the pages given back
    int32_t *keep_sh = give + B;  // committed length
    int32_t *want_sh = keep_sh + B;
    int32_t *held_sh = want_sh + B;  // pages held before, -1 when refused
    cg::cluster_group cluster = cg::this_cluster();
    const int rank = static_cast<int>(cluster.block_rank());
    const int ctas = static_cast<int>(cluster.num_blocks());
    const int page_mask = (1 << P.page_shift) - 1;

    const int head = P.ring_state[0], count = P.ring_state[1];
    const bool ring_ok = head >= 0 && head < P.num_pages && count >= 0 && count <= P.num_pages;
    const int free_pages = ring_ok ? count : 0;
    if (threadIdx.x == 0) granted_sh = 0;
    int bad = ring_ok ? 0 : SSD_DEV_BAD_PAGE;
    uint64_t carry_new = 0, carry_pages = 0;
    for (int base = 0; base < B; base += kPlanThreads) {
        const int b = base + static_cast<int>(threadIdx.x);
        int fresh = 0, held = 0;
        int64_t keep = 0, want = 0;
        bool ok = false;
        if (b < B) {
            fresh = P.new_len[b];
            held = P.held[b];
            keep = P.seq_len[b];
            const int a = P.accept_len ? P.accept_len[b] : -1;
            ok = fresh >= 0 && keep >= 0 && held >= 0 && held <= P.max_blocks;
            if (a >= 0) keep += static_cast<int64_t>(a) + 1;
            if (keep < 0 || keep > 0x7FFFFFFF) keep = P.seq_len[b], ok = false;
            if (fresh < 0) fresh = 0;
            want = (keep + fresh + page_mask) >> P.page_shift;
            if (want > P.max_blocks) ok = false;
        }
        const uint64_t upto = block_scan(static_cast<uint64_t>(fresh), carry_new, red);
        if (b < B && upto > static_cast<uint64_t>(P.cap) && fresh > 0) ok = false;
        if (!ok) want = held;
        // both page sums in one: taken in the high half, given in the low (each below 2^31)
        const uint64_t t = ok && want > held ? static_cast<uint64_t>(want - held) : 0;
        const uint64_t g = ok && want < held ? static_cast<uint64_t>(held - want) : 0;
        const uint64_t pages = block_scan((t << 32) | g, carry_pages, red);
        if (b < B) {
            if (!ok) bad |= SSD_DEV_BAD_LENGTH;
            const uint64_t demand = pages >> 32;
            const bool served = ok && (t == 0 || demand <= static_cast<uint64_t>(free_pages));
            if (ok && !served) bad |= SSD_DEV_NO_PAGES;
            if (served && t) atomicMax(&granted_sh, static_cast<int>(demand));
            cu[b] = static_cast<int>(upto < static_cast<uint64_t>(P.cap) ? upto : static_cast<uint64_t>(P.cap));
            take[b] = static_cast<int>(demand);
            give[b] = static_cast<int>(pages & 0xFFFFFFFFu);
            keep_sh[b] = static_cast<int>(keep);
            want_sh[b] = static_cast<int>(want);
            held_sh[b] = served ? held : -1;
            if (rank == 0) {
                P.cu_new[b + 1] = cu[b];
                P.kv_len[b] = static_cast<int>(served ? keep + fresh : keep);
            }
        }
    }
    if (rank == 0 && threadIdx.x == 0) P.cu_new[0] = 0;
    if (rank == 0) report(P.dev_status, bad);
    // every CTA has read the state; from here on it is written
    if (ctas > 1)
        cluster.sync();
    else
        __syncthreads();

    const int granted = granted_sh;
    const int given = give[B - 1];
    const int tokens = cu[B - 1];
    const int stride = ctas * kPlanThreads;
    const int first = rank * kPlanThreads + static_cast<int>(threadIdx.x);
    // the ring's places are sums of values below num_pages < 2^31: unsigned holds them
    const uint32_t np = static_cast<uint32_t>(P.num_pages);
    for (int i = first; i < granted; i += stride) {
        const int b = first_above(take, B, i);
        const int j = held_sh[b] + i - (b ? take[b - 1] : 0);
        P.block_table[static_cast<int64_t>(b) * P.max_blocks + j] =
            P.ring[(static_cast<uint32_t>(head) + static_cast<uint32_t>(i)) % np];
    }
    if (ring_ok) {
        const uint32_t tail = (static_cast<uint32_t>(head) + static_cast<uint32_t>(count)) % np;
        for (int i = first; i < given; i += stride) {
            const int b = first_above(give, B, i);
            const int j = want_sh[b] + i - (b ? give[b - 1] : 0);
            int32_t *entry = P.block_table + static_cast<int64_t>(b) * P.max_blocks + j;
            P.ring[(tail + static_cast<uint32_t>(i)) % np] = *entry;
            *entry = -1;
        }
    }
    // four tokens at a time, so that their searches and page reads overlap
    bool bad_page = false;
    for (int t0 = first; t0 < P.cap; t0 += stride * kTokens) {
        int pos[kTokens], page[kTokens];
        bool served[kTokens];
#pragma unroll
        for (int k = 0; k < kTokens; ++k) {
            const int t = t0 + k * stride;
            pos[k] = 0, page[k] = -1, served[k] = false;
            if (t >= tokens) continue;
            const int b = first_above(cu, B, t);
            pos[k] = keep_sh[b] + t - (b ? cu[b - 1] : 0);
            const int held = held_sh[b];
            if (held < 0) continue;
            served[k] = true;
            const int block = pos[k] >> P.page_shift;
            // a page taken above is read from the ring again: its table entry may not be there yet
            page[k] = block < held ? P.block_table[static_cast<int64_t>(b) * P.max_blocks + block]
                                   : P.ring[(static_cast<uint32_t>(head) +
                                             static_cast<uint32_t>((b ? take[b - 1] : 0) + block - held)) % np];
        }
#pragma unroll
        for (int k = 0; k < kTokens; ++k) {
            const int t = t0 + k * stride;
            if (t >= P.cap) continue;
            const bool there = page[k] >= 0 && page[k] < P.num_pages;
            bad_page |= served[k] && !there;
            P.slots[t] = there ? (page[k] << P.page_shift) + (pos[k] & page_mask) : -1;
            P.positions[t] = pos[k];
        }
    }
    if (bad_page) report(P.dev_status, SSD_DEV_BAD_PAGE);
    if (rank == 0) {
        for (int b = static_cast<int>(threadIdx.x); b < B; b += kPlanThreads) {
            P.seq_len[b] = keep_sh[b];
            if (held_sh[b] >= 0) P.held[b] = want_sh[b];
        }
        if (threadIdx.x == 0 && ring_ok) {
            P.ring_state[0] = static_cast<int>((static_cast<uint32_t>(head) + static_cast<uint32_t>(granted)) % np);
            P.ring_state[1] = count - granted + given;
        }
    }
}

}  // namespace
}  // namespace ssd

extern "C" int ssd_kv_plan(int32_t *seq_len, const int32_t *accept_len, const int32_t *new_len, int32_t *held, int B,
                           int32_t *block_table, int max_blocks, int32_t *ring, int32_t *ring_state, int num_pages,
                           int page_size, int cap, int32_t *cu_new, int32_t *kv_len, int32_t *slots,
                           int32_t *positions, int32_t *dev_status, void *stream) {
    using namespace ssd;
    if (!seq_len || !new_len || !held || !block_table || !ring || !ring_state || !cu_new || !kv_len ||
        (cap > 0 && (!slots || !positions)))
        return SSD_ERR_INVALID_ARG;
    if (B < 1 || max_blocks < 1 || num_pages < 1 || cap < 0 || !kv_page_size_ok(page_size)) return SSD_ERR_INVALID_ARG;
    if (B > SSD_KV_MAX_B || cap > 0x7FFFFFFF - kTurn || static_cast<int64_t>(B) * max_blocks > 0x7FFFFFFF ||
        static_cast<int64_t>(num_pages) * page_size > 0x7FFFFFFF ||
        static_cast<int64_t>(max_blocks) * page_size > 0x7FFFFFFF)
        return SSD_ERR_UNSUPPORTED;
    const PlanParams P{seq_len,   accept_len,         new_len,     held, B,      block_table, max_blocks, ring,
                       ring_state, num_pages,          log2_of(page_size), cap,  cu_new, kv_len,      slots,      positions,
                       dev_status};
    // More than 48 KB of shared memory, what the kernel has of its own among it, has to be asked for: once for each
    // device, for the largest batch, so that no call lowers what another is about to launch with.
    const size_t dyn = static_cast<size_t>(B) * kSumsBytes;
    static std::atomic<uint64_t> ready{0};
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) {
        cudaGetLastError();
        return SSD_ERR_CUDA;
    }
    const uint64_t bit = 1ull << (dev & 63);
    if (!(ready.load(std::memory_order_relaxed) & bit)) {
        if (cudaFuncSetAttribute(plan_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, SSD_KV_MAX_B * kSumsBytes) !=
            cudaSuccess) {
            cudaGetLastError();
            return SSD_ERR_CUDA;
        }
        ready.fetch_or(bit, std::memory_order_relaxed);
    }
    // one CTA writes 2048 tokens in about the time that a cluster takes to meet twice
    int ctas = 1;
    while (ctas < kPlanCtas && cap > ctas * 2048) ctas *= 2;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(ctas));
    cfg.blockDim = dim3(kPlanThreads);
    cfg.dynamicSmemBytes = dyn;
    cfg.stream = static_cast<cudaStream_t>(stream);
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = static_cast<unsigned>(ctas);
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (cudaLaunchKernelEx(&cfg, plan_kernel, P) != cudaSuccess) {
        cudaGetLastError();
        return SSD_ERR_CUDA;
    }
    return SSD_OK;
}
