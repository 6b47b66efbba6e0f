// ssd_kv_attend.cu -- attention of new tokens over the paged e4m3 cache (sm_103a).
//
//   s_rj = sm_scale <q_r, k8_j> ks(page j),   out_r = sum_j softmax(s_r)_j v8_j vs(page j)
//
// The rows r of one item are the new tokens of a sequence times the query heads that share
// one cache head, kRows of them at most; the item's keys come in tiles of 128.
//
// The 8-bit values go from the cache to the tensor cores as they lie there.  What meets
// them is made of e4m3 digits instead: x = t1 + t2 / 16 (+ t3 / 256), each digit the e4m3
// value nearest to what is left, times 16.  Two digits hold a bf16 query exactly and three
// an fp16 one (down to 2^-14 of the row's largest); a softmax weight is rounded to 2^-8 or
// 2^-12 of itself, as bf16 or fp16 would round it.  The digits of a row are columns of
// their own, so their products are summed apart in fp32 and joined with their weights.
// So there is no conversion pass over the cache, which bounds the call.
//
// The products are taken with the long side first: S^T = K Q^T has the 128 keys as its rows
// and rows x digits as its columns, O^T = V^T P^T the channels.  A few query rows then cost
// a few columns, and both products read K and V in the layout that TMA leaves them in
// (K with its channels, V with its keys as the inner index of the product).
//
// A weight is taken relative to the largest of its own tile, so that its digits' end
// (2^-22 of that) stays below a bf16 step whatever the other tiles hold; the tiles'
// outputs are joined in fp32 registers under the running maximum.
//
// Roles of the warps of a CTA: 0-3 softmax (a thread per key), 4-7 output (a thread per
// channel), 8 TMA, 9 MMA, 10 the queries' digits.  K and V tiles pass through one ring of
// shared-memory slots; S and O are double-buffered in TMEM, weights in shared memory.
//
// Work split.  All tiles of all items form one line, which the CTAs cut into equal
// stretches: ragged lengths and few sequences fill the GPU alike.  A CTA whose stretch ends
// inside an item leaves a partial result (output, maximum, sum) in the workspace, and a
// second kernel, started as the first drains, joins the parts in the order of their keys.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "ssd_kv.h"
#include "ssd_tc.h"

namespace ssd {
namespace {

constexpr int kTile = 128;
constexpr int kAttendWarps = 11;
constexpr int kAttendThreads = 32 * kAttendWarps;
constexpr int kMaxCtas = 320;
constexpr int kMaxRows = 64;
constexpr int kMaxHead = 128;
constexpr int kSeqsInside = 512;   // sequences whose prefix sums every CTA makes itself
constexpr int kMaxPairs = 1 << 18;  // (sequence, row block) pairs of a call with longer items
constexpr float kLog2e = 1.4426950408889634f;

// What a CTA tells the joining kernel: the item whose first part it holds.
struct Join {
    int32_t last_cta;  // -1: nothing to join
    int32_t first_token;
    int32_t row0, rows, head;
    int32_t pad[3];
};

struct Workspace {
    float o[2 * kMaxCtas][kMaxRows][kMaxHead];
    float2 ml[2 * kMaxCtas][kMaxRows];
    Join join[kMaxCtas];
    int32_t pairs;              // of the schedule below
    int32_t sums[kMaxPairs + 1];  // tiles before each pair
    int32_t seq[kMaxPairs];
    int32_t row0[kMaxPairs];
    int32_t start[kMaxCtas + 1];  // pair in which each CTA's stretch starts
};

struct AttendParams {
    const void *q;
    int64_t q_stride;
    const uint8_t *v;
    const float *ks, *vs;
    int num_pages, page_shift, Hq, Hkv, G;
    const int32_t *table;
    int max_blocks;
    const int32_t *cu, *kv_len;
    int B, T, max_new;
    float scale;  // sm_scale * log2(e): scores are held in base 2
    int window;
    int rows_per_item;
    int inside;  // the schedule is made by every CTA in shared memory
    int slots;   // of the K/V ring
    void *out;
    Workspace *ws;
    int32_t *dev_status;
};

struct Seq {
    int first, n, pos0;  // first token, tokens served, position of the first
};

__device__ __forceinline__ Seq load_seq(const AttendParams &P, int b) {
    Seq s;
    s.first = min(max(P.cu[b], 0), P.T);
    const int n = min(max(P.cu[b + 1], s.first), P.T) - s.first;
    s.n = min(n, P.max_new);
    s.pos0 = P.kv_len[b] - n;
    return s;
}

// The keys of rows [row0, row1) of a sequence: [start, stop), in tiles tile0 .. tile0 + tiles.
struct Span {
    int start, stop, tile0, tiles;
};
__device__ __forceinline__ Span key_span(const AttendParams &P, const Seq &s, int row0, int row1) {
    const int low = s.pos0 + row0 / P.G, high = s.pos0 + (row1 - 1) / P.G;
    Span k;
    k.start = P.window > 0 ? max(0, low + 1 - P.window) : 0;
    k.stop = min(high + 1, P.max_blocks << P.page_shift);
    if (k.stop > k.start) {
        k.tile0 = k.start / kTile;
        k.tiles = (k.stop + kTile - 1) / kTile - k.tile0;
    } else {  // nothing to attend to: one tile without keys writes the zeros
        k.start = k.stop = k.tile0 = 0;
        k.tiles = 1;
    }
    return k;
}

__device__ __forceinline__ int first_unit(int64_t cta, int64_t units, int64_t ctas) {
    return static_cast<int>(cta * units / ctas);
}

// One item's part in a CTA's stretch.
struct Part {
    int b, head, row0, rows;
    int first, pos0;      // of the sequence
    int start, stop;      // keys that any row attends to
    int tile, tiles;      // this part's tiles
    bool from_start, to_end;
    int last_cta;         // CTA that holds the item's last tile
};

struct Walk {
    const int32_t *sums, *seq, *row0;
    int unit, end, pair;
    int units, ctas;
    __device__ __forceinline__ bool next(const AttendParams &P, Part &part) {
        if (unit >= end) return false;
        while (sums[pair + 1] <= unit) ++pair;
        const int base = sums[pair], span = sums[pair + 1] - base;
        const int b = P.inside ? pair : seq[pair];
        part.b = b;
        part.row0 = P.inside ? 0 : row0[pair];
        const Seq s = load_seq(P, b);
        part.first = s.first;
        part.pos0 = s.pos0;
        part.rows = min(P.rows_per_item, s.n * P.G - part.row0);
        const Span k = key_span(P, s, part.row0, part.row0 + part.rows);
        part.start = k.start, part.stop = k.stop;
        const int all = span / P.Hkv;  // == k.tiles
        part.head = (unit - base) / all;
        const int done = (unit - base) - part.head * all;
        part.tile = k.tile0 + done;
        part.tiles = min(all - done, end - unit);
        part.from_start = done == 0;
        part.to_end = done + part.tiles == all;
        const int64_t item_end = static_cast<int64_t>(base) + static_cast<int64_t>(part.head + 1) * all;
        part.last_cta = static_cast<int>((item_end * ctas - 1) / units);
        unit += part.tiles;
        return true;
    }
};

// Inclusive sum over the block of one value per thread, plus carry; carry gets the total.
template <int kN>
__device__ __forceinline__ int block_sums(int v, int &carry, int *red) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int t = __shfl_up_sync(0xFFFFFFFFu, v, o);
        if (lane >= o) v += t;
    }
    __syncthreads();
    if (lane == 31) red[warp] = v;
    __syncthreads();
    int before = 0, total = 0;
    for (int w = 0; w < kN / 32; ++w) {
        const int t = red[w];
        if (w < warp) before += t;
        total += t;
    }
    const int r = carry + before + v;
    carry += total;
    return r;
}

__device__ __forceinline__ int last_not_above(const int32_t *sums, int n, int x) {
    int lo = 0, hi = n;  // sums[lo] <= x, and sums[hi] > x where hi < n
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (sums[mid] <= x)
            lo = mid;
        else
            hi = mid;
    }
    return lo;
}

// The schedule of calls whose sequences make several row blocks: one CTA.
constexpr int kScheduleThreads = 1024;
__global__ void __launch_bounds__(kScheduleThreads) schedule_kernel(const __grid_constant__ AttendParams P, int ctas) {
    __shared__ int32_t blocks[SSD_KV_MAX_B + 1];
    __shared__ int red[kScheduleThreads / 32];
    const int tid = threadIdx.x;
    int carry = 0;
    if (tid == 0) blocks[0] = 0;
    for (int base = 0; base < P.B; base += kScheduleThreads) {
        const int b = base + tid;
        int v = 0;
        if (b < P.B) v = (load_seq(P, b).n * P.G + P.rows_per_item - 1) / P.rows_per_item;
        const int sum = block_sums<kScheduleThreads>(v, carry, red);
        if (b < P.B) blocks[b + 1] = sum;
    }
    __syncthreads();
    const int pairs = min(carry, kMaxPairs);
    Workspace &W = *P.ws;
    carry = 0;
    if (tid == 0) W.sums[0] = 0, W.pairs = pairs;
    for (int base = 0; base < pairs; base += kScheduleThreads) {
        const int p = base + tid;
        int v = 0;
        if (p < pairs) {
            const int b = last_not_above(blocks, P.B, p);
            const int row0 = (p - blocks[b]) * P.rows_per_item;
            const Seq s = load_seq(P, b);
            v = key_span(P, s, row0, min(row0 + P.rows_per_item, s.n * P.G)).tiles * P.Hkv;
            W.seq[p] = b;
            W.row0[p] = row0;
        }
        const int sum = block_sums<kScheduleThreads>(v, carry, red);
        if (p < pairs) W.sums[p + 1] = sum;
    }
    __syncthreads();
    const int units = carry, used = min(ctas, units);
    for (int c = tid; c < used; c += kScheduleThreads)
        W.start[c] = last_not_above(W.sums, pairs, first_unit(c, units, used));
}

__device__ __forceinline__ float wide(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float wide(__half x) { return __half2float(x); }
template <class E>
__device__ __forceinline__ E narrow(float x);
template <>
__device__ __forceinline__ __nv_bfloat16 narrow(float x) { return __float2bfloat16(x); }
template <>
__device__ __forceinline__ __half narrow(float x) { return __float2half(x); }

__device__ __forceinline__ float2 floats_of_e4m3x2(uint32_t two) {
    const uint32_t h = halves_of_e4m3x2(two);
    return __half22float2(*reinterpret_cast<const __half2 *>(&h));
}

template <class E>
constexpr int digits_of() {
    return sizeof(E) == 2 && __is_same(E, __half) ? 3 : 2;
}

template <class E_, int kD_, int kR_>
struct Form {
    using E = E_;
    static constexpr int D = kD_, R = kR_;
    static constexpr int kDigits = digits_of<E>();
    static constexpr int N = (R * kDigits + 15) / 16 * 16;              // columns of S and O
    static constexpr int kPitch = N <= 32 ? 32 : (N <= 64 ? 64 : 128);  // bytes of weights per key
    static constexpr int kColumns = 4 * N <= 64 ? 64 : (4 * N <= 128 ? 128 : (4 * N <= 256 ? 256 : 512));
    static constexpr int kCtas = kColumns <= 256 ? 2 : 1;  // per SM
    static constexpr int kSlot = kTile * D;
    static constexpr int kQ = (N * D + 1023) / 1024 * 1024;
    static constexpr int kP = kTile * kPitch;
    static_assert(N <= 128 && 4 * N <= kColumns);
};

// Waits are bounded.  When one runs out, `gave_up` is set and every role goes on through its
// loop without waiting, loading or multiplying, so that all of them reach the end together.
constexpr uint64_t kSliceNs = 50000000;
constexpr int kSlices = 80;  // 4 s
__device__ __forceinline__ void wait_phase(uint64_t *bar, uint32_t parity, int *gave_up) {
    if (mbar_test_wait(bar, parity) || *static_cast<volatile int *>(gave_up)) return;
    for (int i = 0; i < kSlices; ++i) {
        if (mbar_wait_suspend_for(bar, parity, kSliceNs)) return;
        if (*static_cast<volatile int *>(gave_up)) return;
    }
    *static_cast<volatile int *>(gave_up) = 1;
}

constexpr int kRowRing = 4;  // items whose row data may be in use at once
constexpr int kMaxSlots = 12;

template <int R>
struct Shared {
    uint64_t full[kMaxSlots], empty[kMaxSlots];
    uint64_t s_full[2], s_free[2], p_full[2], o_full[2], o_free[2], q_full, q_free, drained;
    float q_factor[kRowRing][R];
    int2 row_keys[kRowRing][R];  // first and last key of a row
    float4 tile_max[2][R];       // of the four softmax warps
    float4 tile_sum[2][R];
    float v_max[2][4];
    float2 joined[2][R];  // factors of the old and the new output
    float final[R];
    int64_t out_at[R];
    uint32_t tmem;
    int nan_met;
    int gave_up;
    int red[kAttendWarps];
};

// Sum over the 32 lanes of each of 8 values; lane l gets the sum of value l / 4.
__device__ __forceinline__ float sums_of_8(const float (&v)[8], int lane) {
    float a[4], b[2];
    const bool h16 = lane & 16, h8 = lane & 8, h4 = lane & 4;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float give = h16 ? v[i] : v[i + 4], keep = h16 ? v[i + 4] : v[i];
        a[i] = keep + __shfl_xor_sync(0xFFFFFFFFu, give, 16);
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const float give = h8 ? a[i] : a[i + 2], keep = h8 ? a[i + 2] : a[i];
        b[i] = keep + __shfl_xor_sync(0xFFFFFFFFu, give, 8);
    }
    float c = (h4 ? b[1] : b[0]) + __shfl_xor_sync(0xFFFFFFFFu, h4 ? b[0] : b[1], 4);
    c += __shfl_xor_sync(0xFFFFFFFFu, c, 2);
    return c + __shfl_xor_sync(0xFFFFFFFFu, c, 1);
}

template <class F>
__global__ void __launch_bounds__(kAttendThreads, F::kCtas)
    attend_kernel(const __grid_constant__ AttendParams P, const __grid_constant__ CUtensorMap k_map,
                  const __grid_constant__ CUtensorMap v_map) {
    using E = typename F::E;
    constexpr int D = F::D, R = F::R, N = F::N, kDigits = F::kDigits, kPitch = F::kPitch;
    extern __shared__ uint8_t raw[];
    uint8_t *base = raw + ((1024 - (smem_addr(raw) & 1023)) & 1023);
    uint8_t *ring = base;
    uint8_t *q_sh = ring + P.slots * F::kSlot;
    uint8_t *p_sh = q_sh + F::kQ;
    Shared<R> &S = *reinterpret_cast<Shared<R> *>(p_sh + 2 * F::kP);
    int32_t *sums_sh = reinterpret_cast<int32_t *>(&S + 1);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int cta = blockIdx.x;
    const int slots = P.slots;

    // ---- schedule -------------------------------------------------------------------
    Walk walk;
    if (P.inside) {
        int carry = 0;
        if (tid == 0) sums_sh[0] = 0;
        for (int b0 = 0; b0 < P.B; b0 += kAttendThreads) {
            const int b = b0 + tid;
            int v = 0;
            if (b < P.B) {
                const Seq s = load_seq(P, b);
                if (s.n > 0) v = key_span(P, s, 0, s.n * P.G).tiles * P.Hkv;
            }
            const int sum = block_sums<kAttendThreads>(v, carry, S.red);
            if (b < P.B) sums_sh[b + 1] = sum;
        }
        __syncthreads();
        walk.sums = sums_sh;
        walk.units = carry;
        walk.seq = walk.row0 = nullptr;
    } else {
        walk.sums = P.ws->sums, walk.seq = P.ws->seq, walk.row0 = P.ws->row0;
        walk.units = P.ws->sums[P.ws->pairs];
    }
    walk.ctas = min(static_cast<int>(gridDim.x), walk.units);
    const bool busy = cta < walk.ctas;
    walk.unit = busy ? first_unit(cta, walk.units, walk.ctas) : 0;
    walk.end = busy ? first_unit(cta + 1, walk.units, walk.ctas) : 0;
    walk.pair = !busy ? 0 : (P.inside ? last_not_above(sums_sh, P.B, walk.unit) : P.ws->start[cta]);

    // Tokens that no item serves get zeros: those behind the last sequence's, and those beyond max_new.
    {
        const int64_t width = static_cast<int64_t>(P.Hq) * D;
        E *out = static_cast<E *>(P.out);
        const int64_t stride = static_cast<int64_t>(gridDim.x) * kAttendThreads;
        const int served = min(max(P.cu[P.B], 0), P.T);
        for (int64_t i = served * width + static_cast<int64_t>(cta) * kAttendThreads + tid; i < P.T * width; i += stride)
            out[i] = narrow<E>(0.f);
        for (int b = cta; b < P.B; b += gridDim.x) {
            const int from = min(max(P.cu[b], 0), P.T), to = min(max(P.cu[b + 1], from), P.T);
            if (to - from <= P.max_new) continue;
            if (tid == 0) report(P.dev_status, SSD_DEV_BAD_LENGTH);
            for (int64_t i = (from + P.max_new) * width + tid; i < to * width; i += kAttendThreads) out[i] = narrow<E>(0.f);
        }
    }

    if (tid == 0) {
        for (int i = 0; i < slots; ++i) mbar_init(&S.full[i], 1), mbar_init(&S.empty[i], 1);
        for (int i = 0; i < 2; ++i) {
            mbar_init(&S.s_full[i], 1);
            mbar_init(&S.s_free[i], 4);
            mbar_init(&S.p_full[i], 4);
            mbar_init(&S.o_full[i], 1);
            mbar_init(&S.o_free[i], 4);
        }
        mbar_init(&S.q_full, 1);
        mbar_init(&S.q_free, 1);
        mbar_init(&S.drained, 1);
        S.nan_met = 0;
        S.gave_up = 0;
        fence_mbar_init();
        P.ws->join[cta].last_cta = -1;
    }
    if (busy && warp == 9) tc::tmem_alloc(&S.tmem, F::kColumns);
    tc::fence_before();
    __syncthreads();
    tc::fence_after();
    if (!busy) return;
    const uint32_t tmem = S.tmem;

    Part part;
    auto wait = [&](uint64_t *bar, int parity) { wait_phase(bar, static_cast<uint32_t>(parity), &S.gave_up); };
    auto gave_up = [&] { return *static_cast<volatile int *>(&S.gave_up) != 0; };
    if (warp < 4) {
        // ---- softmax: one key per thread --------------------------------------------
        int it = 0, item = 0;
        while (walk.next(P, part)) {
            const int ring_row = item % kRowRing;
            ++item;
            const int32_t *table = P.table + static_cast<int64_t>(part.b) * P.max_blocks;
            auto page_of = [&](int j) { return j >= part.start && j < part.stop ? __ldg(table + (j >> P.page_shift)) : -1; };
            auto page_ok = [&](int page) { return page >= 0 && page < P.num_pages; };
            // all rows attend to the keys [common_from, common_to]
            const int low = part.pos0 + part.row0 / P.G, high = part.pos0 + (part.row0 + part.rows - 1) / P.G;
            const int common_to = low, common_from = P.window > 0 ? max(0, high + 1 - P.window) : 0;
            int j = part.tile * kTile + tid;
            int page = page_of(j);
            int page_next = page_of(j + kTile);
            bool ok = page_ok(page);
            float ks = 0.f, vs = 0.f;
            if (ok) {
                ks = __ldg(P.ks + static_cast<int64_t>(page) * P.Hkv + part.head);
                vs = __ldg(P.vs + static_cast<int64_t>(page) * P.Hkv + part.head);
            }
            for (int t = 0; t < part.tiles; ++t, ++it, j += kTile) {
                const int buf = it & 1, phase = (it >> 1) & 1;
                // the next tile's scales and the page of the one after it are under way while this one is worked on
                const bool ok_now = ok;
                const float ks_now = ks, vs_now = vs;
                if (!ok_now && j >= part.start && j < part.stop) report(P.dev_status, SSD_DEV_BAD_PAGE);
                if (t + 1 < part.tiles) {
                    ok = page_ok(page_next);
                    ks = vs = 0.f;
                    if (ok) {
                        ks = __ldg(P.ks + static_cast<int64_t>(page_next) * P.Hkv + part.head);
                        vs = __ldg(P.vs + static_cast<int64_t>(page_next) * P.Hkv + part.head);
                    }
                    page_next = page_of(j + 2 * kTile);
                }
                const float vs_size = ok_now && fabsf(vs_now) <= 3.402823466e38f ? fabsf(vs_now) : 0.f;

                wait(&S.s_full[buf], phase);
                tc::fence_after();
                float s[R];
                const uint32_t at = tmem + buf * N + (static_cast<uint32_t>(warp) << 21);
#pragma unroll
                for (int r = 0; r < R; r += 8) {
                    float d[kDigits][8];
#pragma unroll
                    for (int g = 0; g < kDigits; ++g) tc::tmem_load8(d[g], at + g * R + r);
                    tc::tmem_wait_load(d);
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        s[r + i] = fmaf(d[1][i], 0.0625f, d[0][i]);
                        if (kDigits == 3) s[r + i] = fmaf(d[kDigits - 1][i], 0.00390625f, s[r + i]);
                    }
                }
                tc::fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&S.s_free[buf]);

                const bool partial = !(ok_now && j >= common_from && j <= common_to);
                uint64_t seen = ~0ull;
#pragma unroll
                for (int r = 0; r < R; ++r) s[r] *= ks_now * S.q_factor[ring_row][r];
                if (__any_sync(0xFFFFFFFFu, partial)) {
                    seen = 0;
#pragma unroll
                    for (int r = 0; r < R; ++r) {
                        const int2 keys = S.row_keys[ring_row][r];
                        const bool v = ok_now && j >= keys.x && j <= keys.y;
                        s[r] = v ? s[r] : -INFINITY;
                        seen |= static_cast<uint64_t>(v) << r;
                    }
                }
                // the output warps have read what this buffer held two tiles ago
                if (it >= 2) wait(&S.o_free[buf], phase ^ 1);
                float mine[(R + 31) / 32];
#pragma unroll
                for (int r = 0; r < R; ++r) {
                    const float m = tc::warp_max(s[r]);
                    if ((r & 31) == lane) mine[r >> 5] = m;
                }
                float *max_sh = reinterpret_cast<float *>(S.tile_max[buf]);
#pragma unroll
                for (int r = 0; r < (R + 31) / 32; ++r)
                    if (r * 32 + lane < R) max_sh[(r * 32 + lane) * 4 + warp] = mine[r];
                const float v_top = tc::warp_max(vs_size);
                if (lane == 0) S.v_max[buf][warp] = v_top;
                tc::named_barrier(1, 128);

                // weights p = 2^(s - max); their digits carry p vs / v_ref times 256, v_ref a power of two
                const float v_all = fmaxf(fmaxf(S.v_max[buf][0], S.v_max[buf][1]), fmaxf(S.v_max[buf][2], S.v_max[buf][3]));
                const uint32_t v_exp = min(max(__float_as_uint(v_all) >> 23, 8u), 254u);  // 2^(v_exp - 126) > v_all
                const float v_scale = __uint_as_float((254u + 7u - v_exp) << 23);           // 2^(134 - v_exp) = 256 / 2^(v_exp - 126)
                float f = vs_now * v_scale;
                if (!(fabsf(vs_now) <= 3.402823466e38f)) f = __int_as_float(0x7FC00000);
                uint8_t *p_at = p_sh + buf * F::kP;
                uint32_t words[kDigits][R / 4];
                float *sum_sh = reinterpret_cast<float *>(S.tile_sum[buf]);
#pragma unroll
                for (int r0 = 0; r0 < R; r0 += 8) {
                    float p[8];
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const float4 m4 = S.tile_max[buf][r0 + i];
                        float m = fmaxf(fmaxf(m4.x, m4.y), fmaxf(m4.z, m4.w));
                        m = m == -INFINITY ? 0.f : m;
                        p[i] = ex2(s[r0 + i] - m);
                    }
                    float w[8];
#pragma unroll
                    for (int i = 0; i < 8; ++i) w[i] = (seen >> (r0 + i)) & 1 ? p[i] * f : 0.f;
#pragma unroll
                    for (int g = 0; g < kDigits; ++g) {
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            const uint32_t a = e4m3x2(w[4 * h], w[4 * h + 1]), b = e4m3x2(w[4 * h + 2], w[4 * h + 3]);
                            words[g][r0 / 4 + h] = a | (b << 16);
                            if (g + 1 < kDigits) {
                                const float2 fa = floats_of_e4m3x2(a), fb = floats_of_e4m3x2(b);
                                w[4 * h] = (w[4 * h] - fa.x) * 16.f;
                                w[4 * h + 1] = (w[4 * h + 1] - fa.y) * 16.f;
                                w[4 * h + 2] = (w[4 * h + 2] - fb.x) * 16.f;
                                w[4 * h + 3] = (w[4 * h + 3] - fb.y) * 16.f;
                            }
                        }
                    }
                    const float sum = sums_of_8(p, lane);
                    if ((lane & 3) == 0) sum_sh[(r0 + lane / 4) * 4 + warp] = sum;
                }
                // columns g * R + r of this key's row
                constexpr int kWords = kDigits * R / 4;
                const uint32_t *flat = &words[0][0];
#pragma unroll
                for (int c = 0; c < (kWords + 3) / 4; ++c) {
                    uint4 v;
                    v.x = flat[4 * c];
                    v.y = 4 * c + 1 < kWords ? flat[4 * c + 1] : 0u;
                    v.z = 4 * c + 2 < kWords ? flat[4 * c + 2] : 0u;
                    v.w = 4 * c + 3 < kWords ? flat[4 * c + 3] : 0u;
                    *reinterpret_cast<uint4 *>(p_at + tc::swizzled<kPitch>(tid, c)) = v;
                }
                if (partial) {
                    // A weight of 0 times NaN is NaN: values that no row, or not every row, attends to are
                    // cleared where that could happen.  NaN that some rows do attend to is put back by the output warps.
                    const int slot = (2 * it + 1) % slots, round = (2 * it + 1) / slots;
                    wait(&S.full[slot], round & 1);
                    uint4 *row = reinterpret_cast<uint4 *>(ring + slot * F::kSlot + tid * D);
                    if (seen == 0) {
#pragma unroll
                        for (int c = 0; c < D / 16; ++c) row[c] = make_uint4(0, 0, 0, 0);
                    } else {
                        bool met = false;
#pragma unroll
                        for (int c = 0; c < D / 16; ++c) {
                            uint4 w4 = row[c];
                            uint32_t *w = &w4.x;
                            bool here = false;
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                // a byte is NaN iff its low seven bits are all set
                                const uint32_t nan = ((w[e] & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u;
                                if (nan) {
                                    here = true;
                                    w[e] &= ~((nan >> 7) * 0xFFu);
                                }
                            }
                            if (here) row[c] = w4, met = true;
                        }
                        if (met) atomicExch(&S.nan_met, 1);
                    }
                }
                tc::fence_async_shared();
                __syncwarp();
                if (lane == 0) mbar_arrive(&S.p_full[buf]);
            }
        }
    } else if (warp < 8) {
        // ---- output: one channel per thread -------------------------------------------
        const int ch = tid - 128;
        int it = 0;
        while (walk.next(P, part)) {
            float acc[R];
#pragma unroll
            for (int r = 0; r < R; ++r) acc[r] = 0.f;
            float m_run = -INFINITY, l_run = 0.f;  // of row ch
            for (int t = 0; t < part.tiles; ++t, ++it) {
                const int buf = it & 1, phase = (it >> 1) & 1;
                wait(&S.p_full[buf], phase);
                if (ch < R) {
                    const float4 m4 = S.tile_max[buf][ch], l4 = S.tile_sum[buf][ch];
                    const float m = fmaxf(fmaxf(m4.x, m4.y), fmaxf(m4.z, m4.w));
                    const float v_all =
                        fmaxf(fmaxf(S.v_max[buf][0], S.v_max[buf][1]), fmaxf(S.v_max[buf][2], S.v_max[buf][3]));
                    const uint32_t v_exp = min(max(__float_as_uint(v_all) >> 23, 8u), 254u);
                    const float v_unit = __uint_as_float((v_exp - 7u) << 23);  // 2^(v_exp - 134)
                    const float m_new = fmaxf(m_run, m);
                    const float ref = m_new == -INFINITY ? 0.f : m_new;
                    const float old = ex2(m_run - ref), now = ex2(m - ref);
                    l_run = l_run * old + ((l4.x + l4.y) + (l4.z + l4.w)) * (m == -INFINITY ? 1.f : now);
                    m_run = m_new;
                    S.joined[buf][ch] = make_float2(old, now * v_unit);
                }
                tc::named_barrier(2, 128);
                wait(&S.o_full[buf], phase);
                tc::fence_after();
                const uint32_t at = tmem + (2 + buf) * N + (static_cast<uint32_t>(warp - 4) << 21);
#pragma unroll
                for (int r = 0; r < R; r += 8) {
                    float d[kDigits][8];
#pragma unroll
                    for (int g = 0; g < kDigits; ++g) tc::tmem_load8(d[g], at + g * R + r);
                    tc::tmem_wait_load(d);
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        float o = fmaf(d[1][i], 0.0625f, d[0][i]);
                        if (kDigits == 3) o = fmaf(d[kDigits - 1][i], 0.00390625f, o);
                        const float2 f = S.joined[buf][r + i];
                        acc[r + i] = fmaf(o, f.y, acc[r + i] * f.x);
                    }
                }
                tc::fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&S.o_free[buf]);
            }
            if (*static_cast<volatile int *>(&S.nan_met) && ch < D) {
                // rare: NaN among values that only some rows attend to, read again from the cache
                const int high = part.pos0 + (part.row0 + part.rows - 1) / P.G, low = part.pos0 + part.row0 / P.G;
                const int from = max(part.start, part.tile * kTile), to = min(part.stop, (part.tile + part.tiles) * kTile);
                for (int j = from; j < to; ++j) {
                    if (j <= low && (P.window == 0 || j > high - P.window)) continue;
                    const int page = P.table[static_cast<int64_t>(part.b) * P.max_blocks + (j >> P.page_shift)];
                    if (page < 0 || page >= P.num_pages) continue;
                    const int64_t row = ((static_cast<int64_t>(page) * P.Hkv + part.head) << P.page_shift) +
                                        (j & ((1 << P.page_shift) - 1));
                    if ((P.v[row * D + ch] & 0x7F) != 0x7F) continue;
#pragma unroll
                    for (int r = 0; r < R; ++r) {
                        const int pos = part.pos0 + (part.row0 + r) / P.G;
                        if (j <= pos && (P.window == 0 || j > pos - P.window)) acc[r] = __int_as_float(0x7FC00000);
                    }
                }
            }
            const bool whole = part.from_start && part.to_end;
            if (whole) {
                if (ch < R) {
                    const int row = part.row0 + ch;
                    const int token = part.first + row / P.G, head = part.head * P.G + row % P.G;
                    S.final[ch] = l_run == 0.f ? 0.f : 1.f / l_run;
                    S.out_at[ch] = (static_cast<int64_t>(token) * P.Hq + head) * D;
                }
                tc::named_barrier(2, 128);
                if (ch < D) {
                    E *out = static_cast<E *>(P.out) + ch;
#pragma unroll
                    for (int r = 0; r < R; ++r)
                        if (r < part.rows) out[S.out_at[r]] = narrow<E>(acc[r] * S.final[r]);
                }
                tc::named_barrier(2, 128);
            } else {
                const int slot = 2 * cta + (part.from_start ? 1 : 0);
                if (ch < R) P.ws->ml[slot][ch] = make_float2(m_run, l_run);
                if (ch < D)
#pragma unroll
                    for (int r = 0; r < R; ++r)
                        if (r < part.rows) P.ws->o[slot][r][ch] = acc[r];
                if (part.from_start && ch == 0) {
                    Join jn{};
                    jn.last_cta = part.last_cta;
                    jn.first_token = part.first;
                    jn.row0 = part.row0;
                    jn.rows = part.rows;
                    jn.head = part.head;
                    P.ws->join[cta] = jn;
                }
            }
        }
    } else if (warp == 8) {
        // ---- TMA: K and V of each tile, one slot each -----------------------------------
        int it = 0;
        int issued = 0;
        const int pages_per_tile = kTile >> P.page_shift;
        while (walk.next(P, part)) {
            const int32_t *table = P.table + static_cast<int64_t>(part.b) * P.max_blocks;
            // each lane holds one of 32 consecutive pages, and the one 32 later
            const int page_of_tile = part.tile * pages_per_tile;
            auto load_page = [&](int i) {
                const int j = i << P.page_shift;
                return j < part.stop && j + (1 << P.page_shift) > part.start ? __ldg(table + i) : -1;
            };
            int held = load_page(page_of_tile + lane), later = load_page(page_of_tile + 32 + lane);
            int held_from = page_of_tile;
            for (int t = 0; t < part.tiles; ++t, ++it) {
                const int p0 = page_of_tile + t * pages_per_tile;
                if (p0 - held_from >= 32) {
                    held = later, held_from += 32;
                    later = load_page(held_from + 32 + lane);
                }
                const int page = __shfl_sync(0xFFFFFFFFu, held, (p0 - held_from + (lane & (pages_per_tile - 1))) & 31);
                const bool load = lane < pages_per_tile && page >= 0 && page < P.num_pages;
                const int n = __popc(__ballot_sync(0xFFFFFFFFu, load));
                const uint32_t bytes = static_cast<uint32_t>(n) * static_cast<uint32_t>(D << P.page_shift);
                const int row = (page * P.Hkv + part.head) << P.page_shift;
#pragma unroll
                for (int what = 0; what < 2; ++what) {
                    const int x = 2 * it + what, slot = x % slots, round = x / slots;
                    if (round > 0) wait(&S.empty[slot], (round - 1) & 1);
                    const bool go = __all_sync(0xFFFFFFFFu, !gave_up());
                    if (go && lane == 0) mbar_arrive_expect_tx(&S.full[slot], bytes);
                    __syncwarp();
                    if (go && load)
                        tc::tma_load_2d(ring + slot * F::kSlot + lane * (D << P.page_shift), what ? &v_map : &k_map, 0, row,
                                        &S.full[slot]);
                    issued = go ? x + 1 : issued;
                }
            }
        }
        if (gave_up())  // the copies under way still have to land before the CTA ends
            for (int x = max(0, issued - slots); x < issued; ++x)
                for (int i = 0; i < kSlices && !mbar_wait_suspend_for(&S.full[x % slots], (x / slots) & 1, kSliceNs); ++i) {
                }
    } else if (warp == 9) {
        // ---- MMA ----------------------------------------------------------------------
        if (lane == 0) {
            constexpr uint32_t kShapeS = tc::mma_shape(N, false, false), kShapeO = tc::mma_shape(N, true, true);
            const uint64_t q_desc = tc::matrix_desc(q_sh, D);
            int it = 0, item = 0;
            auto output_of = [&](int i) {  // O^T = V^T P^T of tile i
                const int buf = i & 1, phase = (i >> 1) & 1;
                const int slot = (2 * i + 1) % slots, round = (2 * i + 1) / slots;
                wait(&S.full[slot], round & 1);
                wait(&S.p_full[buf], phase);
                if (i >= 2) wait(&S.o_free[buf], phase ^ 1);
                if (gave_up()) return;
                tc::fence_after();
                const uint64_t v_desc = tc::matrix_desc(ring + slot * F::kSlot, D);
                const uint64_t p_desc = tc::matrix_desc(p_sh + buf * F::kP, kPitch);
#pragma unroll
                for (int k = 0; k < kTile / 32; ++k)
                    tc::mma_e4m3(tmem + (2 + buf) * N, v_desc + k * (32 * D >> 4), p_desc + k * (32 * kPitch >> 4), kShapeO, k > 0);
                tc::mma_commit(&S.o_full[buf]);
                tc::mma_commit(&S.empty[slot]);
            };
            while (walk.next(P, part)) {
                wait(&S.q_full, item & 1);
                ++item;
                for (int t = 0; t < part.tiles; ++t, ++it) {
                    const int buf = it & 1, phase = (it >> 1) & 1;
                    const int slot = (2 * it) % slots, round = (2 * it) / slots;
                    wait(&S.full[slot], round & 1);
                    if (it >= 2) wait(&S.s_free[buf], phase ^ 1);
                    if (gave_up()) continue;
                    tc::fence_after();
                    const uint64_t k_desc = tc::matrix_desc(ring + slot * F::kSlot, D);
#pragma unroll
                    for (int k = 0; k < D / 32; ++k)  // 32 channels further inside the swizzled rows
                        tc::mma_e4m3(tmem + buf * N, k_desc + k * 2, q_desc + k * 2, kShapeS, k > 0);
                    tc::mma_commit(&S.s_full[buf]);
                    tc::mma_commit(&S.empty[slot]);
                    if (t == part.tiles - 1) tc::mma_commit(&S.q_free);
                    if (it > 0) output_of(it - 1);
                }
            }
            if (it > 0) output_of(it - 1);
            if (gave_up()) {  // what was issued still has to end before the CTA does
                tc::mma_commit(&S.drained);
                for (int i = 0; i < kSlices && !mbar_wait_suspend_for(&S.drained, 0, kSliceNs); ++i) {
                }
            }
        }
        __syncwarp();
    } else {
        // ---- the queries' digits --------------------------------------------------------
        constexpr int kPer = D / 32;  // channels per lane
        constexpr int kBatch = 8;     // rows in flight
        int item = 0;
        while (walk.next(P, part)) {
            const int ring_row = item % kRowRing;
#pragma unroll 1
            for (int r0 = 0; r0 < R; r0 += kBatch) {
                float x[kBatch][kPer];
#pragma unroll
                for (int i = 0; i < kBatch; ++i) {
                    const int row = part.row0 + r0 + i;
                    const bool there = r0 + i < part.rows;
                    const E *q = static_cast<const E *>(P.q) + (part.first + row / P.G) * P.q_stride +
                                 static_cast<int64_t>(part.head * P.G + row % P.G) * D + lane * kPer;
#pragma unroll
                    for (int c = 0; c < kPer; c += 2) {
                        uint32_t two = 0;
                        if (there) two = __ldg(reinterpret_cast<const uint32_t *>(q + c));
                        x[i][c] = wide(reinterpret_cast<const E *>(&two)[0]);
                        x[i][c + 1] = wide(reinterpret_cast<const E *>(&two)[1]);
                    }
                }
                if (r0 == 0 && item > 0) wait(&S.q_free, (item - 1) & 1);
#pragma unroll
                for (int i = 0; i < kBatch; ++i) {
                    const int r = r0 + i;
                    float top = 0.f;
                    bool odd = false;
#pragma unroll
                    for (int c = 0; c < kPer; ++c) {
                        odd |= !(fabsf(x[i][c]) <= 3.402823466e38f);
                        top = fmaxf(top, fabsf(x[i][c]));
                    }
                    top = tc::warp_max(top);
                    odd = __any_sync(0xFFFFFFFFu, odd);
                    // the largest is brought into [128, 256): k = 7 - its exponent
                    const int e = static_cast<int>(__float_as_uint(top) >> 23);
                    const int k = top == 0.f ? 0 : min(134 - e, 126);
                    const float up = __uint_as_float(static_cast<uint32_t>(127 + k) << 23);
                    uint32_t digit[kDigits];
                    float left[kPer];
#pragma unroll
                    for (int c = 0; c < kPer; ++c) left[c] = x[i][c] * up;
#pragma unroll
                    for (int g = 0; g < kDigits; ++g) {
                        digit[g] = 0;
#pragma unroll
                        for (int c = 0; c < kPer; c += 2) {
                            const uint32_t two = e4m3x2(left[c], left[c + 1]);
                            const float2 f = floats_of_e4m3x2(two);
                            left[c] = (left[c] - f.x) * 16.f;
                            left[c + 1] = (left[c + 1] - f.y) * 16.f;
                            digit[g] |= two << (8 * c);
                        }
                        const int at = tc::swizzled<D>(g * R + r, lane * kPer / 16) + (lane * kPer) % 16;
                        if (kPer == 4)
                            *reinterpret_cast<uint32_t *>(q_sh + at) = digit[g];
                        else
                            *reinterpret_cast<uint16_t *>(q_sh + at) = static_cast<uint16_t>(digit[g]);
                    }
                    if (lane == 0) {
                        const bool there = r < part.rows;
                        const int pos = part.pos0 + (part.row0 + r) / P.G;
                        // 2^-k in two steps: k reaches 126 and -120
                        float f = P.scale * __uint_as_float(static_cast<uint32_t>(127 - k) << 23);
                        if (odd) f = __int_as_float(0x7FC00000);
                        S.q_factor[ring_row][r] = there ? f : 0.f;
                        S.row_keys[ring_row][r] =
                            there ? make_int2(P.window > 0 ? pos + 1 - P.window : 0, pos) : make_int2(0, -1);
                    }
                }
            }
            tc::fence_async_shared();
            __syncwarp();
            if (lane == 0) mbar_arrive(&S.q_full);
            ++item;
        }
    }
    if (tid == 0 && gave_up()) report(P.dev_status, SSD_DEV_TIMEOUT);
    tc::fence_before();
    __syncthreads();
    tc::fence_after();
    if (warp == 9) tc::tmem_free(tmem, F::kColumns);
}

// Joins the parts of the items that several CTAs share: one warp per row.
template <class E, int D>
__global__ void __launch_bounds__(128) join_kernel(const __grid_constant__ AttendParams P) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int cta = blockIdx.x, lane = threadIdx.x & 31;
    const int r = blockIdx.y * 4 + (threadIdx.x >> 5);
    const Join jn = P.ws->join[cta];
    if (jn.last_cta < 0 || r >= jn.rows) return;
    const int parts = jn.last_cta - cta + 1;
    auto slot = [&](int i) { return i == 0 ? 2 * cta + 1 : 2 * (cta + i); };
    float top = -INFINITY;
    for (int i = lane; i < parts; i += 32) top = fmaxf(top, P.ws->ml[slot(i)][r].x);
    top = tc::warp_max(top);
    const float ref = top == -INFINITY ? 0.f : top;
    constexpr int kPer = D / 32;
    float acc[kPer], total = 0.f;
#pragma unroll
    for (int c = 0; c < kPer; ++c) acc[c] = 0.f;
    for (int i0 = 0; i0 < parts; i0 += 32) {
        float w = 0.f, l = 0.f;
        if (i0 + lane < parts) {
            const float2 ml = P.ws->ml[slot(i0 + lane)][r];
            w = ex2(ml.x - ref);
            l = ml.y * (ml.x == -INFINITY ? 1.f : w);
        }
        const int n = min(32, parts - i0);
#pragma unroll 8
        for (int i = 0; i < n; ++i) {
            const float wi = __shfl_sync(0xFFFFFFFFu, w, i);
            total += __shfl_sync(0xFFFFFFFFu, l, i);
            const float *o = &P.ws->o[slot(i0 + i)][r][lane * kPer];
#pragma unroll
            for (int c = 0; c < kPer; ++c) acc[c] = fmaf(wi, o[c], acc[c]);
        }
    }
    const float inv = total == 0.f ? 0.f : 1.f / total;
    const int row = jn.row0 + r;
    E *out = static_cast<E *>(P.out) +
             (static_cast<int64_t>(jn.first_token + row / P.G) * P.Hq + jn.head * P.G + row % P.G) * D + lane * kPer;
#pragma unroll
    for (int c = 0; c < kPer; ++c) out[c] = narrow<E>(acc[c] * inv);
}

struct Device {
    int sms = 0;
    int smem_sm = 0, smem_cta = 0;
};
int device_limits(Device *d) {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&d->sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&d->smem_sm, cudaDevAttrMaxSharedMemoryPerMultiprocessor, dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&d->smem_cta, cudaDevAttrMaxSharedMemoryPerBlockOptin, dev) != cudaSuccess) {
        cudaGetLastError();
        return SSD_ERR_CUDA;
    }
    return SSD_OK;
}

template <class F>
int attend_launch(AttendParams P, const CUtensorMap &k_map, const CUtensorMap &v_map, const Device &dev, cudaStream_t stream) {
    auto *kernel = attend_kernel<F>;
    const int fixed = 1024 + F::kQ + 2 * F::kP + static_cast<int>(sizeof(Shared<F::R>)) + (kSeqsInside + 1) * 4;
    const int room = F::kCtas == 2 ? dev.smem_sm / 2 - 1024 : dev.smem_cta;
    int slots = (room - fixed) / F::kSlot;
    if (slots > kMaxSlots) slots = kMaxSlots;
    if (slots < 3) return SSD_ERR_UNSUPPORTED;
    const int dyn = fixed + slots * F::kSlot;
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, dyn) != cudaSuccess) {
        cudaGetLastError();
        return SSD_ERR_CUDA;
    }
    P.slots = slots;
    P.rows_per_item = F::R;
    P.inside = static_cast<int64_t>(P.max_new) * P.G <= F::R && P.B <= kSeqsInside;
    int ctas = dev.sms * F::kCtas;
    if (ctas > kMaxCtas) ctas = kMaxCtas;
    if (!P.inside) {
        if (static_cast<int64_t>(P.T) * P.G / F::R + P.B > kMaxPairs) return SSD_ERR_UNSUPPORTED;
        schedule_kernel<<<1, kScheduleThreads, 0, stream>>>(P, ctas);
        if (launched() != SSD_OK) return SSD_ERR_CUDA;
    }
    kernel<<<static_cast<unsigned>(ctas), kAttendThreads, static_cast<size_t>(dyn), stream>>>(P, k_map, v_map);
    if (launched() != SSD_OK) return SSD_ERR_CUDA;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(ctas), (F::R + 3) / 4);
    cfg.blockDim = dim3(128);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (cudaLaunchKernelEx(&cfg, join_kernel<typename F::E, F::D>, P) != cudaSuccess) {
        cudaGetLastError();
        return SSD_ERR_CUDA;
    }
    return SSD_OK;
}

// Rows of an item: the fewest that hold the tokens of a sequence, so that few rows cost few columns.
template <class E, int D>
int attend_dispatch(const AttendParams &P, const CUtensorMap &k, const CUtensorMap &v, const Device &dev, cudaStream_t s) {
    const int64_t rows = static_cast<int64_t>(P.max_new) * P.G;
    if (rows <= 8) return attend_launch<Form<E, D, 8>>(P, k, v, dev, s);
    if (rows <= 16) return attend_launch<Form<E, D, 16>>(P, k, v, dev, s);
    if (rows <= 32 || digits_of<E>() == 3) return attend_launch<Form<E, D, 32>>(P, k, v, dev, s);
    if constexpr (digits_of<E>() == 2) return attend_launch<Form<E, D, 64>>(P, k, v, dev, s);
    return SSD_ERR_UNSUPPORTED;
}

}  // namespace
}  // namespace ssd

extern "C" size_t ssd_kv_workspace_size(void) { return (sizeof(ssd::Workspace) + 255) / 256 * 256; }

extern "C" int ssd_kv_attend(const void *q, int dtype, int64_t q_stride, const void *k_cache, const void *v_cache,
                             const float *k_scale, const float *v_scale, int num_pages, int page_size, int Hq, int Hkv,
                             int D, const int32_t *block_table, int max_blocks, const int32_t *cu_new,
                             const int32_t *kv_len, int B, int T, int max_new, float sm_scale, int window, void *out,
                             void *workspace, size_t workspace_bytes, int32_t *dev_status, void *stream) {
    using namespace ssd;
    if (dtype != SSD_BF16 && dtype != SSD_F16) return SSD_ERR_DTYPE;
    if (B < 1 || T < 0 || max_new < 1 || num_pages < 1 || max_blocks < 1 || Hkv < 1 || Hq < 1 || Hq % Hkv != 0 ||
        window < 0 || !kv_page_size_ok(page_size) || (D != 64 && D != 128))
        return SSD_ERR_INVALID_ARG;
    if (!(sm_scale == sm_scale) || sm_scale - sm_scale != 0.f) return SSD_ERR_INVALID_ARG;
    if (!k_cache || !v_cache || !k_scale || !v_scale || !block_table || !cu_new || !kv_len || (T > 0 && (!q || !out)))
        return SSD_ERR_INVALID_ARG;
    if (!aligned(k_cache, 16) || !aligned(v_cache, 16)) return SSD_ERR_INVALID_ARG;
    if (T > 0 && (!aligned(q, 16) || !aligned(out, 16))) return SSD_ERR_INVALID_ARG;
    if (T > 1 && (q_stride < static_cast<int64_t>(Hq) * D || q_stride % 8 != 0)) return SSD_ERR_INVALID_ARG;
    if (!workspace || !aligned(workspace, 256) || workspace_bytes < ssd_kv_workspace_size()) return SSD_ERR_WORKSPACE;
    if (static_cast<int64_t>(num_pages) * page_size > 0x7FFFFFFF ||
        static_cast<int64_t>(num_pages) * Hkv > 0x7FFFFFFF / page_size ||
        static_cast<int64_t>(B) * max_blocks > 0x7FFFFFFF || static_cast<int64_t>(max_blocks) * page_size > 0x7FFFFFFF / 2 ||
        B > SSD_KV_MAX_B)
        return SSD_ERR_UNSUPPORTED;
    // tiles of all items, which the schedule counts in 32 bits
    const int64_t row_blocks = static_cast<int64_t>(T < 1 ? 1 : T) * (Hq / Hkv) / 8 + B;
    if (row_blocks * Hkv > 0x7FFFFFFF / (static_cast<int64_t>(max_blocks) * page_size / kTile + 2)) return SSD_ERR_UNSUPPORTED;
    if (T == 0) return SSD_OK;
    AttendParams P{};
    P.q = q;
    P.q_stride = q_stride;
    P.v = static_cast<const uint8_t *>(v_cache);
    P.ks = k_scale, P.vs = v_scale;
    P.num_pages = num_pages;
    P.page_shift = log2_of(page_size);
    P.Hq = Hq, P.Hkv = Hkv, P.G = Hq / Hkv;
    P.table = block_table;
    P.max_blocks = max_blocks;
    P.cu = cu_new, P.kv_len = kv_len;
    P.B = B, P.T = T, P.max_new = max_new < T ? max_new : T;
    P.scale = sm_scale * kLog2e;
    P.window = window;
    P.out = out;
    P.ws = static_cast<Workspace *>(workspace);
    P.dev_status = dev_status;
    Device dev;
    if (device_limits(&dev) != SSD_OK) return SSD_ERR_CUDA;
    CUtensorMap k_map, v_map;
    const uint64_t rows = static_cast<uint64_t>(num_pages) * Hkv * page_size;
    if (!tc::encode_rows(&k_map, k_cache, rows, D, page_size) || !tc::encode_rows(&v_map, v_cache, rows, D, page_size))
        return SSD_ERR_CUDA;
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (dtype == SSD_BF16)
        return D == 64 ? attend_dispatch<__nv_bfloat16, 64>(P, k_map, v_map, dev, s)
                       : attend_dispatch<__nv_bfloat16, 128>(P, k_map, v_map, dev, s);
    return D == 64 ? attend_dispatch<__half, 64>(P, k_map, v_map, dev, s)
                   : attend_dispatch<__half, 128>(P, k_map, v_map, dev, s);
}
