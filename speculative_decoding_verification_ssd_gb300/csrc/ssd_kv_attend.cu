// ssd_kv_attend.cu -- attention of new tokens over the paged e4m3 cache (sm_103a).
//
//   s_rj = sm_scale <q_r, k8_j> ks(page j),   out_r = sum_j softmax(s_r)_j v8_j vs(page j)
//
// The rows r of one item are the new tokens of a sequence times the query heads that share
// one cache head, 32 or 64 of them at most.
//
// The 8-bit values go from the cache to the tensor cores as they lie there: no pass converts
// the cache, whose bytes bound the calls of few rows.  What meets them is made of e4m3
// digits: x = t1 + t2 (+ t3), each the e4m3 value nearest to what the ones before leave.
// * A query row is scaled by a power of two that brings its largest channel into [128, 256).
//   Two digits then hold a bf16 channel exactly down to 2^-9 of the largest, three an fp16
//   one down to 2^-6; smaller ones are off by 2^-17 of the largest at most.
// * A softmax weight is scaled to 256 at most.  Two digits (bf16) round it by 2^-9 of itself
//   (after a half, by 2^-11), three (fp16) by 2^-14, less than half a step of those types; they
//   end at 2^-18 and 2^-23 of the largest weight of the step (fp16's second and third digits are of 32 times what is left
//   and summed apart).  A weight is taken relative to the largest of its own step of 256 (or
//   128) keys, so that a long flat tail is not lost next to a large weight elsewhere; the
//   steps' outputs are joined in fp32 registers under the running maximum.
//
// The products are taken with the long side first: S^T = K Q^T has 128 keys as its rows and
// the item's rows as its columns, O^T = V^T P^T the channels.  A few query rows then cost a
// few columns, and both products read K and V in the layout that TMA leaves them in (K with
// its channels, V with its keys as the inner index of the product).
//
// Roles of the warps of a CTA: 0-7 softmax, in two groups that take steps in turn (a thread
// per key of each tile); 8-11 output (a thread per channel); 12 TMA; 13 MMA; 14 the queries'
// digits; 15 the scout, which walks the items and looks up pages and scales ahead of the
// others.  K and V pass through one ring of shared-memory slots in the order of their use;
// S and O are double-buffered in TMEM, the weights in shared memory.  One warp issues all
// MMAs: two warps that issued S and O apart gained 1%, and a run of them ended in a launch
// failure that reading did not explain.
//
// Work split.  All steps of all items form one line, which the CTAs (one to an SM) cut into
// equal stretches: ragged lengths and few sequences fill the GPU alike.  A CTA whose stretch
// ends inside an item leaves a partial result (output, maximum, sum) in the workspace, and
// the CTA that brings an item's last part joins them all.
//
// What bounds it (one GB300, copy rate 6764 GB/s; calls captured into graphs, L2 flushed).
// One token a sequence: HBM (64 sequences of 8000 to 8191 keys, 8 heads of 128: 171 us, 6.2
// TB/s; of 3 to 8191 keys 101 us, 5.3 TB/s: the shorter the items, the more of them a CTA
// starts).  20 rows: the same (117 us, 4.6 TB/s; fp16 140 us).  36 rows and more: the softmax
// groups (4 sequences of 90 to 131 thousand keys: 201 us, 4.5 TB/s), whose chains of TMEM
// reads, conversions and stores leave half the issue cycles empty and DRAM at 57%.  Prompts the
// same, with next to no bytes (202 us).  Measured on the way, for 64 sequences and 20 rows: loops
// unrolled over the rows missed the instruction cache on 41% of requests (404 us, against
// 265 rolled); a query warp that took four rows at a time held up every change of item (265,
// against 142); 24 warps with two to each 32 keys were slower (178, against 131).
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <atomic>

#include "ssd_kv.h"
#include "ssd_tc.h"

namespace ssd {
namespace {

constexpr int kTile = 128;
constexpr int kMaxCtas = 160;
constexpr int kMaxRows = 64;
constexpr int kMaxHead = 128;
constexpr int kSeqsInside = 256;   // sequences whose prefix sums every CTA makes itself
constexpr int kMaxPairs = 1 << 18;  // (sequence, row block) pairs of a call with longer items
constexpr float kLog2e = 1.4426950408889634f;

struct Workspace {
    float o[2 * kMaxCtas][kMaxRows][kMaxHead];
    float2 ml[2 * kMaxCtas][kMaxRows];
    int32_t arrived[kMaxCtas];  // parts of the item that starts in each CTA; left at 0
    int32_t pairs;              // of the schedule below
    int32_t sums[kMaxPairs + 1];  // steps before each pair
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
    int step_shift;  // log2 of the keys of one step
    int item_cost;   // what starting an item counts in the split, in steps
    int inside;  // the schedule is made by every CTA in shared memory
    int most_pairs;  // (sequence, row block) pairs that T tokens of B sequences can make: what the host's limits are of
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

// The keys of rows [row0, row1) of a sequence: [start, stop), in steps step0 .. step0 + steps.
struct Span {
    int start, stop, step0, steps;
};
__device__ __forceinline__ Span key_span(const AttendParams &P, const Seq &s, int row0, int row1) {
    const int low = s.pos0 + row0 / P.G, high = s.pos0 + (row1 - 1) / P.G;
    Span k;
    k.start = P.window > 0 ? max(0, low + 1 - P.window) : 0;
    k.stop = min(high + 1, P.max_blocks << P.page_shift);
    if (k.stop > k.start) {
        k.step0 = k.start >> P.step_shift;
        k.steps = ((k.stop - 1) >> P.step_shift) + 1 - k.step0;
    } else {  // nothing to attend to: one step without keys writes the zeros
        k.start = k.stop = k.step0 = 0;
        k.steps = 1;
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
    int step, steps;      // this part's
    int first_cta, parts;  // CTAs that the item is cut over: first_cta and the parts - 1 after it
};

struct Walk {
    const int32_t *sums, *seq, *row0;
    int unit, end, pair;
    int units, ctas;
    // A CTA's units are steps, after item_cost units for the start of each item.
    __device__ __forceinline__ bool next(const AttendParams &P, Part &part) {
        for (;;) {
            if (unit >= end) return false;
            while (sums[pair + 1] <= unit) ++pair;
            const int base = sums[pair], all = (sums[pair + 1] - base) / P.Hkv;
            const int head = (unit - base) / all, done = (unit - base) - head * all - P.item_cost;
            if (done < 0) {
                unit -= done;
                continue;
            }
            const int b = P.inside ? pair : seq[pair];
            part.b = b;
            part.row0 = P.inside ? 0 : row0[pair];
            const Seq s = load_seq(P, b);
            part.first = s.first;
            part.pos0 = s.pos0;
            part.rows = min(P.rows_per_item, s.n * P.G - part.row0);
            const Span k = key_span(P, s, part.row0, part.row0 + part.rows);
            part.start = k.start, part.stop = k.stop;
            part.head = head;
            part.step = k.step0 + done;
            part.steps = min(k.steps - done, end - unit);
            const int64_t item = static_cast<int64_t>(base) + static_cast<int64_t>(head) * all;
            part.first_cta = static_cast<int>(((item + P.item_cost + 1) * ctas - 1) / units);
            part.parts = static_cast<int>(((item + all) * ctas - 1) / units) - part.first_cta + 1;
            unit += part.steps;
            return true;
        }
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
    const int pairs = min(carry, P.most_pairs);  // more only of a cu_new that falls
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
            v = (key_span(P, s, row0, min(row0 + P.rows_per_item, s.n * P.G)).steps + P.item_cost) * P.Hkv;
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

// Two halves as e4m3, the low one in the low byte; rounding and range as e4m3x2.
__device__ __forceinline__ uint32_t e4m3x2_of_halves(__half2 v) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(r) : "r"(*reinterpret_cast<const uint32_t *>(&v)));
    return r;
}

template <class E>
constexpr int digits_of() {
    return sizeof(E) == 2 && __is_same(E, __half) ? 3 : 2;
}

template <class E_, int kD_, int kR_>
struct Form {
    using E = E_;
    static constexpr int D = kD_, R = kR_;  // channels, most rows of an item
    static constexpr int kDigits = digits_of<E>();
    static constexpr int N = R;  // columns set aside for S and O
    // tiles of 128 keys in one step: two, unless the weights' digits then leave too few slots for K and V
    static constexpr int kSub = R > 32 && kDigits == 3 && D == 128 ? 1 : 2;
    static constexpr int kStep = kSub * kTile;
    // Starting an item (its queries' digits, a drained pipeline) takes 2.3 us, a step of up to 32 rows 1.4 us and
    // one of 64 rows 3 us.
    static constexpr int kItemCost = R > 32 ? 1 : 2;
    // O has two columns for each row.  Two digits of a weight (bf16) are the two columns of one product: an
    // MMA of few columns takes the time of its 128 rows of V (39 clocks at 16 columns, 47 at 64, 62 at 128),
    // so one of both digits costs little more than one of each.  Of three digits (fp16) the second and third
    // share a column; they are of 32 times what is left.
    static constexpr bool kBoth = kDigits == 2;
    static constexpr float kFine = kBoth ? 1.f : 32.f;
    static constexpr int kPasses = kBoth ? 1 : kDigits;   // products of O
    static constexpr int kPitch = kBoth ? 2 * R : R;      // bytes of a key's weights in one product
    static constexpr int kUsed = (2 * kSub + 4) * N;
    static constexpr int kColumns = kUsed <= 256 ? 256 : 512;
    static constexpr int kSlot = kStep * D;
    static constexpr int kQ = N * D;           // one digit of the queries
    static constexpr int kP = kStep * kPitch;  // weights of one product
    static_assert((R == 32 || R == 64) && kUsed <= kColumns && kQ % 1024 == 0 && kP % 1024 == 0);
};

constexpr int kAttendWarps = 16;  // softmax 2 x 4, output 4, TMA, MMA, queries, scout
constexpr int kAttendThreads = 32 * kAttendWarps;
constexpr int kSteps = 6;    // steps that the scout may be ahead
constexpr int kItems = 6;    // items whose row data may be in use at once (steps s - 4 to s, when each is an item of its own)
constexpr int kMaxSlots = 12;
constexpr int kSharedBytes = 227 * 1024;  // of one CTA
constexpr int kConsumers = 4 + 4 + 3;  // warps that read one step: a softmax group, output, TMA, MMA, queries

// One step of a CTA's stretch: up to kStep keys of one item.
struct Step {
    int32_t live;       // 0: the stretch has ended
    int32_t first, last;  // of its part
    int32_t plain;      // every row attends to every key, and every page is there
    int32_t odd;        // a value scale is not finite
    int32_t key0, subs;  // first key, tiles in use
    int32_t start, stop;  // keys that some row attends to
    int32_t common_from, common_to;  // ... and that every row does
    int32_t there;      // bit p: page p is there
    int32_t item;       // row data of kItems
    int32_t first_cta, parts;  // of the item
    int32_t seq, head, row0, rows, token0, pos0;
    int32_t part_key0;  // first key of the part
    float v_unit;       // what the weights' value scales were divided by
    int32_t page[16];
    float2 scale[16];   // of the keys, and of the values over v_unit
};

template <int R>
struct Shared {
    uint64_t full[kMaxSlots], empty[kMaxSlots];
    uint64_t step_full[kSteps], step_free[kSteps];
    uint64_t s_full[2], s_free[2], p_full[2], o_full[2], o_free[2], q_full, q_free, drained;
    Step step[kSteps];
    alignas(16) float q_factor[kItems][R];
    int32_t row_last[kItems][R];  // last key of a row
    alignas(16) float step_max[4][4][R];  // of the last steps and the four warps of a softmax group
    alignas(16) float row_max[8][R];      // a softmax warp's copy of what they come to
    float4 step_sum[2][R];
    float2 joined[2][R];  // factors of the old and the new output
    float final[R];
    int64_t out_at[R];
    uint32_t tmem;
    int nan_met[kItems];  // NaN among an item's values that only some rows attend to, cleared by the output warps
    int gave_up;
    int highest;  // place in the ring of the last copy issued
    int last_part;
    int red[kAttendWarps];
};

// Waits are bounded by a number of polls (each may suspend the thread for a while: seconds in all, far
// more than any step takes).  When one runs out, `gave_up` is set and every role leaves its loop without
// waiting for the others; barriers that a whole group shares are met by all of it or by none.
constexpr int kPolls = 1 << 22;
__device__ __forceinline__ bool wait_phase(uint64_t *bar, uint32_t parity, volatile int *gave_up) {
    int polls = 0;
    while (!mbar_try_wait(bar, parity)) {
        if (*gave_up || ++polls == kPolls) {
            *gave_up = 1;
            return false;
        }
    }
    return true;
}
// The same for what has to end whether or not a wait ran out.
__device__ __forceinline__ void drain_phase(uint64_t *bar, uint32_t parity) {
    for (int i = 0; i < kPolls && !mbar_try_wait(bar, parity); ++i) {
    }
}

// Whether a row whose last key is `last` attends to key j >= 0.
__device__ __forceinline__ bool attends(const AttendParams &P, int last, int j) {
    return j <= last && (P.window == 0 || j > last - P.window);
}

// Reduces each of kN values over the 32 lanes: kN / 32 results per lane (one where kN < 32), of the
// values from lane * kN / 32 on.  Each round halves the values by trading halves with a partner lane.
struct SumOf {
    __device__ __forceinline__ float operator()(float a, float b) const { return a + b; }
};
template <int kN, class Op>
__device__ __forceinline__ void reduce_lanes(float (&v)[kN], int lane, Op op) {
    int n = kN;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        if (n > 1) {
            n >>= 1;
            const bool high = lane & o;
#pragma unroll
            for (int i = 0; i < kN / 2; ++i) {
                if (i >= n) break;
                const float give = high ? v[i] : v[i + n], keep = high ? v[i + n] : v[i];
                v[i] = op(keep, __shfl_xor_sync(0xFFFFFFFFu, give, o));
            }
        } else {
            v[0] = op(v[0], __shfl_xor_sync(0xFFFFFFFFu, v[0], o));
        }
    }
}

// Shared memory besides the ring of K and V slots, which gets the rest.
template <class F>
constexpr int kFixedBytes = 1024 + F::kDigits * F::kQ + 2 * F::kPasses * F::kP + static_cast<int>(sizeof(Shared<F::R>)) + (kSeqsInside + 1) * 4;
template <class F>
constexpr int kSlots = (kSharedBytes - kFixedBytes<F>) / F::kSlot < kMaxSlots ? (kSharedBytes - kFixedBytes<F>) / F::kSlot : kMaxSlots;

template <class F>
__global__ void __launch_bounds__(kAttendThreads, 1)
    attend_kernel(const __grid_constant__ AttendParams P, const __grid_constant__ CUtensorMap k_map,
                  const __grid_constant__ CUtensorMap v_map) {
    using E = typename F::E;
    constexpr int D = F::D, R = F::R, N = F::N, kDigits = F::kDigits, kPitch = F::kPitch, kSub = F::kSub;
    constexpr uint32_t kAll = 0xFFFFFFFFu;
    extern __shared__ uint8_t raw[];
    uint8_t *base = raw + ((1024 - (smem_addr(raw) & 1023)) & 1023);
    uint8_t *ring = base;
    uint8_t *q_sh = ring + kSlots<F> * F::kSlot;
    uint8_t *p_sh = q_sh + kDigits * F::kQ;
    Shared<R> &S = *reinterpret_cast<Shared<R> *>(p_sh + 2 * F::kPasses * F::kP);
    int32_t *sums_sh = reinterpret_cast<int32_t *>(&S + 1);
    const int tid = threadIdx.x, lane = tid & 31;
    const int warp = __shfl_sync(kAll, tid >> 5, 0);
    const int cta = blockIdx.x;
    constexpr int slots = kSlots<F>;

    if (tid == 0) tc::prefetch_map(&k_map), tc::prefetch_map(&v_map);
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
                if (s.n > 0) v = (key_span(P, s, 0, s.n * P.G).steps + P.item_cost) * P.Hkv;
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
            const int first = P.cu[b], next = P.cu[b + 1], keys = P.kv_len[b];
            const int from = min(max(first, 0), P.T), to = min(max(next, from), P.T);
            // a length counts where tokens are there to attend over it
            const bool fits = first >= 0 && next >= first && next <= P.T &&
                              (to == from || (keys >= 0 && keys <= P.max_blocks << P.page_shift));
            if (tid == 0 && (!fits || to - from > P.max_new)) report(P.dev_status, SSD_DEV_BAD_LENGTH);
            for (int64_t i = (from + P.max_new) * width + tid; i < to * width; i += kAttendThreads) out[i] = narrow<E>(0.f);
        }
    }

    if (tid == 0) {
        for (int i = 0; i < slots; ++i) mbar_init(&S.full[i], 1), mbar_init(&S.empty[i], 1);
        for (int i = 0; i < kSteps; ++i) mbar_init(&S.step_full[i], 1), mbar_init(&S.step_free[i], kConsumers);
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
        for (int i = 0; i < kItems; ++i) S.nan_met[i] = 0;
        S.gave_up = 0;
        fence_mbar_init();
    }
    if (busy && warp == 13) tc::tmem_alloc(&S.tmem, F::kColumns);
    tc::fence_before();
    __syncthreads();
    tc::fence_after();
    if (!busy) return;
    const uint32_t tmem = S.tmem;

    auto wait = [&](uint64_t *bar, int parity) { return wait_phase(bar, static_cast<uint32_t>(parity), &S.gave_up); };
    auto gave_up = [&] { return *static_cast<volatile int *>(&S.gave_up) != 0; };
    // Whether step s is there and not the end, the same for a warp's lanes.  After a wait that ran out its fields may be
    // anything, and are not used.
    auto open_step = [&](int s) {
        const bool came = wait(&S.step_full[s % kSteps], (s / kSteps) & 1);
        return !__any_sync(kAll, !came || !S.step[s % kSteps].live);
    };
    auto close_step = [&](int s) {
        __syncwarp();
        if (lane == 0) mbar_arrive(&S.step_free[s % kSteps]);
    };
    // The ring's order is the order in which the MMA warp uses it: K0 K1 K2 V0 K3 V1 ...
    auto place_of_k = [](int s) { return s < 2 ? s : 2 * s - 2; };
    auto place_of_v = [](int s) { return 2 * s + 3; };

    if (warp < 8) {
        // ---- softmax: one key of each tile per thread; the two groups take steps in turn ----
        const int group = warp >> 2, quad = warp & 3, key = tid & 127;
        const uint32_t s_at = tmem + group * (kSub * N) + (static_cast<uint32_t>(quad) << 21);
        uint8_t *p_at = p_sh + group * (F::kPasses * F::kP);
        // Rows pass in chunks of eight, twice: for the largest scores, then for the weights.  S is read from TMEM
        // each time: the loops stay small enough for the instruction cache (unrolled over 32 rows, instruction
        // fetches took 7 of every 18 stalled cycles), and no row count needs registers of its own.
        for (int it = group;; it += 2) {
            const int phase = (it >> 1) & 1;
            float(&max_sh)[4][R] = S.step_max[it & 3];
            float *sum_sh = reinterpret_cast<float *>(S.step_sum[group]);
            const bool stop = !open_step(it);
            const Step &st = S.step[it % kSteps];
            const int item = stop ? 0 : st.item, chunks = (st.rows + 7) >> 3;
            const float *q_factor = S.q_factor[item];
            const bool plain = st.plain, odd = st.odd;
            float ks[kSub], f[kSub];
            bool there[kSub];
#pragma unroll
            for (int u = 0; u < kSub; ++u) {
                const int page = (u * kTile + key) >> P.page_shift;
                const float2 sc = st.scale[page];
                ks[u] = sc.x, f[u] = sc.y;
                there[u] = (st.there >> page) & 1;
            }
            const int key0 = st.key0 + key;
            auto fetch = [&](int r0, float(&s)[kSub][8]) {
#pragma unroll
                for (int u = 0; u < kSub; ++u) tc::tmem_load(s[u], s_at + u * N + r0);
            };
            // Scores of eight rows, without the rows' own factors; `next` holds what was fetched of them and then
            // gets the following rows under way.
            auto scores = [&](int r0, float(&next)[kSub][8], float(&s)[kSub][8]) {
                tc::tmem_wait_load(next);
#pragma unroll
                for (int u = 0; u < kSub; ++u)
#pragma unroll
                    for (int i = 0; i < 8; ++i) s[u][i] = next[u][i];
                if (r0 + 8 < chunks * 8) fetch(r0 + 8, next);
#pragma unroll
                for (int u = 0; u < kSub; ++u)
#pragma unroll
                    for (int i = 0; i < 8; ++i) s[u][i] *= ks[u];
                if (!plain) {
#pragma unroll
                    for (int u = 0; u < kSub; ++u)
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            s[u][i] = there[u] && attends(P, S.row_last[item][r0 + i], key0 + u * kTile) ? s[u][i] : -INFINITY;
                        }
                }
            };
            if (!stop) {
                wait(&S.s_full[group], phase);
                tc::fence_after();
                // largest score of each row: over the thread's keys, the warp's lanes, the group's warps
                float next[kSub][8];
                fetch(0, next);
#pragma unroll 1
                for (int c = 0; c < chunks; ++c) {
                    float s[kSub][8];
                    scores(c * 8, next, s);
                    if (kSub == 2) {
#pragma unroll
                        for (int i = 0; i < 8; ++i) s[0][i] = fmaxf(s[0][i], s[kSub - 1][i]);
                    }
                    // (2.3 clocks a reduction; the shuffles that trade halves take 8 a row)
                    float mine = 0.f;
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const float m = tc::warp_max(s[0][i]);
                        mine = lane == i ? m : mine;
                    }
                    if (lane < 8) max_sh[quad][c * 8 + lane] = mine * q_factor[c * 8 + lane];
                }
            }
            if (tc::barrier_or(1 + group, 128, stop || gave_up())) break;
            // the weights this group wrote before have been used
            if (it >= 2) wait(&S.o_free[group], phase ^ 1);

            // weights 2^(score - largest), their sums over the keys, and the digits of weight x value scale (<= 256)
            // each lane joins the four warps' maxima of one row in 32; without a key the largest is -inf, and
            // 2^(-inf + 1e30) is 0 all the same
            float *row_max = S.row_max[warp];
#pragma unroll
            for (int i = 0; i < R / 32; ++i) {
                const int r = i * 32 + lane;
                row_max[r] = fmaxf(fmaxf(fmaxf(max_sh[0][r], max_sh[1][r]), fmaxf(max_sh[2][r], max_sh[3][r])), -1e30f);
            }
            __syncwarp();
            float next[kSub][8];
            fetch(0, next);
#pragma unroll 1
            for (int c = 0; c < chunks; ++c) {
                const int r0 = c * 8;
                float s[kSub][8], sums[8], qfs[8], ms[8];
                scores(r0, next, s);
#pragma unroll
                for (int i = 0; i < 8; i += 4) {
                    const float4 q4 = *reinterpret_cast<const float4 *>(q_factor + r0 + i);
                    qfs[i] = q4.x, qfs[i + 1] = q4.y, qfs[i + 2] = q4.z, qfs[i + 3] = q4.w;
                    const float4 m4 = *reinterpret_cast<const float4 *>(row_max + r0 + i);
                    ms[i] = m4.x, ms[i + 1] = m4.y, ms[i + 2] = m4.z, ms[i + 3] = m4.w;
                }
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float m = ms[i], qf = qfs[i];
                    sums[i] = 0.f;
#pragma unroll
                    for (int u = 0; u < kSub; ++u) {
                        s[u][i] = ex2(fmaf(s[u][i], qf, -m));
                        sums[i] += s[u][i];
                    }
                }
                reduce_lanes(sums, lane, SumOf());
                if (lane % 4 == 0) sum_sh[(r0 + lane / 4) * 4 + quad] = sums[0];
#pragma unroll
                for (int u = 0; u < kSub; ++u) {
#pragma unroll
                    for (int i = 0; i < 8; ++i) s[u][i] *= f[u];
                    if (odd && !plain) {  // 0 times a scale that is not finite, for rows that do not attend to the key
#pragma unroll 1
                        for (int i = 0; i < 8; ++i) {
                            if (there[u] && attends(P, S.row_last[item][r0 + i], key0 + u * kTile)) continue;
#pragma unroll
                            for (int e = 0; e < 8; ++e)
                                if (e == i) s[u][e] = 0.f;
                        }
                    }
                    uint32_t words[kDigits][2];
                    if (F::kBoth) {
                        // Two digits hold 2^-8 of a weight, so a half (2^-11) does for the product with the value scale,
                        // rounded once; what is left of it after the first digit is exact.
#pragma unroll
                        for (int h = 0; h < 4; ++h) {
                            const __half2 w = __floats2half2_rn(s[u][2 * h], s[u][2 * h + 1]);
                            const uint32_t a = e4m3x2_of_halves(w);
                            const uint32_t back = halves_of_e4m3x2(a);
                            const uint32_t b = e4m3x2_of_halves(__hsub2(w, *reinterpret_cast<const __half2 *>(&back)));
                            words[0][h / 2] = h % 2 == 0 ? a : words[0][h / 2] | (a << 16);
                            words[1][h / 2] = h % 2 == 0 ? b : words[1][h / 2] | (b << 16);
                        }
                    } else {
#pragma unroll
                        for (int g = 0; g < kDigits; ++g)
#pragma unroll
                            for (int h = 0; h < 2; ++h) {
                                float *w = &s[u][4 * h];
                                const uint32_t a = e4m3x2(w[0], w[1]), b = e4m3x2(w[2], w[3]);
                                words[g][h] = a | (b << 16);
                                if (g + 1 < kDigits) {
                                    const float2 fa = floats_of_e4m3x2(a), fb = floats_of_e4m3x2(b);
                                    const float up = g == 0 ? F::kFine : 1.f;
                                    w[0] = (w[0] - fa.x) * up, w[1] = (w[1] - fa.y) * up;
                                    w[2] = (w[2] - fb.x) * up, w[3] = (w[3] - fb.y) * up;
                                }
                            }
                    }
#pragma unroll
                    for (int g = 0; g < kDigits; ++g) {
                        const int at = F::kBoth ? g * chunks + c : c;  // in units of 8 bytes of the key's row
                        *reinterpret_cast<uint2 *>(p_at + (F::kBoth ? 0 : g * F::kP) +
                                                   tc::swizzled<kPitch>(u * kTile + key, at >> 1) + (at & 1) * 8) =
                            make_uint2(words[g][0], words[g][1]);
                    }
                }
            }
            tc::fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&S.s_free[group]);
            if (!plain) {
                // A weight of 0 times NaN is NaN: values that no row, or not every row, attends to are
                // cleared of it.  NaN that some rows do attend to is put back by the output warps.
                const int place = place_of_v(it), slot = place % slots;
                wait(&S.full[slot], (place / slots) & 1);
#pragma unroll
                for (int u = 0; u < kSub; ++u) {
                    const int j = key0 + u * kTile;
                    const bool seen = there[u] && j >= st.start && j < st.stop;
                    if (u >= st.subs || (seen && j >= st.common_from && j <= st.common_to)) continue;
                    uint4 *row = reinterpret_cast<uint4 *>(ring + slot * F::kSlot + (u * kTile + key) * D);
                    if (!seen) {
#pragma unroll 1
                        for (int c = 0; c < D / 16; ++c) row[c] = make_uint4(0, 0, 0, 0);
                    } else {
                        bool met = false;
#pragma unroll 1
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
                        if (met) atomicExch(&S.nan_met[item], 1);
                    }
                }
            }
            tc::fence_async_shared();
            __syncwarp();
            if (lane == 0) mbar_arrive(&S.p_full[group]);
            close_step(it);
        }
    } else if (warp < 12) {
        // ---- output: one channel per thread -------------------------------------------
        const int ch = tid - 256, quad = warp & 3;
        float acc[R];
        float m_run = -INFINITY, l_run = 0.f;  // of row ch
#pragma unroll
        for (int r = 0; r < R; ++r) acc[r] = 0.f;
        for (int it = 0;; ++it) {
            const int buf = it & 1, phase = (it >> 1) & 1;
            const bool stop = !open_step(it);
            const Step &st = S.step[it % kSteps];
            if (!stop) wait(&S.p_full[buf], phase);
            if (!stop && ch < st.rows) {
                const float(&ms)[4][R] = S.step_max[it & 3];
                const float4 l4 = S.step_sum[buf][ch];
                const float m = fmaxf(fmaxf(ms[0][ch], ms[1][ch]), fmaxf(ms[2][ch], ms[3][ch]));
                const float m_new = fmaxf(m_run, m);
                const float ref = m_new == -INFINITY ? 0.f : m_new;
                const float old = ex2(m_run - ref), now = ex2(m - ref);
                l_run = l_run * old + ((l4.x + l4.y) + (l4.z + l4.w)) * (m == -INFINITY ? 1.f : now);
                m_run = m_new;
                S.joined[buf][ch] = make_float2(old, now * st.v_unit);
            }
            if (tc::barrier_or(3, 128, stop || gave_up())) break;
            wait(&S.o_full[buf], phase);
            tc::fence_after();
            const uint32_t at = tmem + 2 * kSub * N + buf * (2 * N) + (static_cast<uint32_t>(quad) << 21);
            const int rows = st.rows, second = F::kBoth ? (rows + 7) & ~7 : N;
#pragma unroll
            for (int r0 = 0; r0 < R; r0 += 8) {
                if (r0 < rows) {
                    float o[2][8];
                    tc::tmem_load(o[0], at + r0);
                    tc::tmem_load(o[1], at + second + r0);
                    tc::tmem_wait_load(o);
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const float2 f = S.joined[buf][r0 + i];
                        acc[r0 + i] = fmaf(fmaf(o[1][i], 1.f / F::kFine, o[0][i]), f.y, acc[r0 + i] * f.x);
                    }
                }
            }
            tc::fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&S.o_free[buf]);
            if (st.last) {
                const bool nan_met = *static_cast<volatile int *>(&S.nan_met[st.item]) != 0;
                if (nan_met && ch < D) {
                    // rare: NaN among values that only some rows attend to, read again from the cache
                    const int from = max(st.start, st.part_key0), to = min(st.stop, st.key0 + F::kStep);
                    for (int j = from; j < to; ++j) {
                        if (j >= st.common_from && j <= st.common_to) continue;
                        const int page = P.table[static_cast<int64_t>(st.seq) * P.max_blocks + (j >> P.page_shift)];
                        if (page < 0 || page >= P.num_pages) continue;
                        const int64_t row = ((static_cast<int64_t>(page) * P.Hkv + st.head) << P.page_shift) +
                                            (j & ((1 << P.page_shift) - 1));
                        if ((P.v[row * D + ch] & 0x7F) != 0x7F) continue;
#pragma unroll
                        for (int r = 0; r < R; ++r) {
                            if (attends(P, S.row_last[st.item][r], j)) acc[r] = __int_as_float(0x7FC00000);
                        }
                    }
                }
                if (st.parts == 1) {
                    if (ch < R) {
                        const int row = st.row0 + ch;
                        const int token = st.token0 + row / P.G, head = st.head * P.G + row % P.G;
                        S.final[ch] = l_run == 0.f ? 0.f : 1.f / l_run;
                        S.out_at[ch] = (static_cast<int64_t>(token) * P.Hq + head) * D;
                    }
                    tc::named_barrier(3, 128);
                    if (ch < D) {
                        E *out = static_cast<E *>(P.out) + ch;
#pragma unroll
                        for (int r = 0; r < R; ++r)
                            if (r < st.rows) out[S.out_at[r]] = narrow<E>(acc[r] * S.final[r]);
                    }
                    tc::named_barrier(3, 128);
                } else {
                    // The part goes to the workspace; the CTA that brings the last one joins them, in the order of
                    // their keys whoever that is.
                    Workspace &W = *P.ws;
                    const int rows = st.rows, parts = st.parts, first_cta = st.first_cta;
                    auto slot_of = [&](int c) { return 2 * c + (c == first_cta ? 1 : 0); };
                    const int slot = slot_of(cta);
                    if (ch < rows) __stcg(&W.ml[slot][ch], make_float2(m_run, l_run));
                    if (ch < D)
#pragma unroll
                        for (int r = 0; r < R; ++r)
                            if (r < rows) __stcg(&W.o[slot][r][ch], acc[r]);
                    __threadfence();
                    tc::named_barrier(3, 128);
                    if (ch == 0) S.last_part = atomicAdd(&W.arrived[first_cta], 1) == parts - 1;
                    tc::named_barrier(3, 128);
                    if (S.last_part) {
                        __threadfence();
                        if (ch == 0) W.arrived[first_cta] = 0;
                        // each part's share of a row, in place of its maximum
                        constexpr int kHeld = 8;
                        if (ch < rows) {
                            float2 ml[kHeld];
#pragma unroll
                            for (int i = 0; i < kHeld; ++i)
                                ml[i] = i < parts ? __ldcg(&W.ml[slot_of(first_cta + i)][ch]) : make_float2(-INFINITY, 0.f);
                            float top = -INFINITY, total = 0.f;
#pragma unroll
                            for (int i = 0; i < kHeld; ++i) top = fmaxf(top, ml[i].x);
#pragma unroll 8
                            for (int i = kHeld; i < parts; ++i) top = fmaxf(top, __ldcg(&W.ml[slot_of(first_cta + i)][ch]).x);
                            const float ref = top == -INFINITY ? 0.f : top;
                            auto weight = [&](float2 v) { return v.y * (v.x == -INFINITY ? 1.f : ex2(v.x - ref)); };
#pragma unroll
                            for (int i = 0; i < kHeld; ++i) total += weight(ml[i]);
#pragma unroll 8
                            for (int i = kHeld; i < parts; ++i) total += weight(__ldcg(&W.ml[slot_of(first_cta + i)][ch]));
                            const float inv = total == 0.f ? 0.f : 1.f / total;
#pragma unroll
                            for (int i = 0; i < kHeld; ++i)
                                if (i < parts) __stcg(&W.ml[slot_of(first_cta + i)][ch].x, ex2(ml[i].x - ref) * inv);
#pragma unroll 8
                            for (int i = kHeld; i < parts; ++i) {
                                float2 *at = &W.ml[slot_of(first_cta + i)][ch];
                                __stcg(&at->x, ex2(__ldcg(at).x - ref) * inv);
                            }
                            const int row = st.row0 + ch;
                            S.out_at[ch] = (static_cast<int64_t>(st.token0 + row / P.G) * P.Hq + st.head * P.G + row % P.G) * D;
                        }
                        tc::named_barrier(3, 128);
                        if (ch < D) {
                            E *out = static_cast<E *>(P.out) + ch;
                            constexpr int kRows = 8;  // of four parts in flight
#pragma unroll 1
                            for (int r0 = 0; r0 < rows; r0 += kRows) {
                                float sum[kRows];
#pragma unroll
                                for (int k = 0; k < kRows; ++k) sum[k] = 0.f;
#pragma unroll 1
                                for (int i = 0; i < parts; i += 4) {
                                    float w[4][kRows], o[4][kRows];
#pragma unroll
                                    for (int e = 0; e < 4; ++e) {
                                        const int from = slot_of(first_cta + min(i + e, parts - 1));
#pragma unroll
                                        for (int k = 0; k < kRows; ++k) {
                                            const int row = min(r0 + k, rows - 1);
                                            w[e][k] = i + e < parts ? __ldcg(&W.ml[from][row].x) : 0.f;
                                            o[e][k] = i + e < parts ? __ldcg(&W.o[from][row][ch]) : 0.f;
                                        }
                                    }
#pragma unroll
                                    for (int e = 0; e < 4; ++e)
#pragma unroll
                                        for (int k = 0; k < kRows; ++k) sum[k] = fmaf(w[e][k], o[e][k], sum[k]);
                                }
#pragma unroll
                                for (int k = 0; k < kRows; ++k)
                                    if (r0 + k < rows) out[S.out_at[r0 + k]] = narrow<E>(sum[k]);
                            }
                        }
                        tc::named_barrier(3, 128);
                    }
                }
                // all four warps have read it, at a barrier since; the next item of this number starts after this step is closed
                if (nan_met && ch == 0) S.nan_met[st.item] = 0;
#pragma unroll
                for (int r = 0; r < R; ++r) acc[r] = 0.f;
                m_run = -INFINITY, l_run = 0.f;
            }
            close_step(it);
        }
    } else if (warp == 12) {
        // ---- TMA ------------------------------------------------------------------------
        int highest = -1;
        auto load = [&](int s, int place, const CUtensorMap *map) {
            const Step &st = S.step[s % kSteps];
            const int slot = place % slots, round = place / slots;
            if (round > 0) wait(&S.empty[slot], (round - 1) & 1);
            if (__any_sync(kAll, gave_up())) return;
            const bool mine = lane < 16 && ((st.there >> lane) & 1);
            const int bytes = __popc(static_cast<uint32_t>(st.there)) * (D << P.page_shift);
            if (lane == 0) mbar_arrive_expect_tx(&S.full[slot], static_cast<uint32_t>(bytes));
            __syncwarp();
            if (mine)
                tc::tma_load_2d(ring + slot * F::kSlot + lane * (D << P.page_shift), map, 0,
                                (st.page[lane] * P.Hkv + st.head) << P.page_shift, &S.full[slot]);
            highest = max(highest, place);
        };
        int n = 0;
        for (;; ++n) {
            if (!open_step(n)) break;
            const Step &st = S.step[n % kSteps];
            load(n, place_of_k(n), &k_map);
            if (n >= 2) {
                load(n - 2, place_of_v(n - 2), &v_map);
                close_step(n - 2);
            }
        }
        for (int s = max(0, n - 2); s < n; ++s) {
            load(s, place_of_v(s), &v_map);
            close_step(s);
        }
        if (lane == 0) S.highest = highest;
    } else if (warp == 13) {
        // ---- MMA ------------------------------------------------------------------------
        const uint64_t ring_k = tc::matrix_desc(ring, D), q_desc = tc::matrix_desc(q_sh, D);
        const uint64_t p_desc = tc::matrix_desc(p_sh, kPitch);
        auto output_of = [&](int s, int subs, int columns) {  // O^T = V^T P^T of step s
            const int buf = s & 1, phase = (s >> 1) & 1;
            const int place = place_of_v(s), slot = place % slots;
            wait(&S.full[slot], (place / slots) & 1);
            wait(&S.p_full[buf], phase);
            if (s >= 2) wait(&S.o_free[buf], phase ^ 1);
            if (__any_sync(kAll, gave_up())) return;
            tc::fence_after();
            const uint32_t shape = tc::mma_shape(columns, true, true);
            if (tc::elect_one()) {
#pragma unroll 1
                for (int u = 0; u < subs; ++u) {
#pragma unroll 1
                    for (int g = 0; g < F::kPasses; ++g)
#pragma unroll
                        for (int k = 0; k < kTile / 32; ++k)
                            tc::mma_e4m3(tmem + 2 * kSub * N + buf * (2 * N) + (!F::kBoth && g > 0 ? N : 0),
                                         ring_k + ((slot * F::kSlot + (u * kTile + k * 32) * D) >> 4),
                                         p_desc + (((buf * F::kPasses + g) * F::kP + (u * kTile + k * 32) * kPitch) >> 4), shape,
                                         u + k + (g == 2) > 0);
                }
                tc::mma_commit(&S.o_full[buf]);
                tc::mma_commit(&S.empty[slot]);
            }
            __syncwarp();
        };
        // tiles and columns of the last step, and of the one before
        int n = 0, items = 0, subs_1 = 0, subs_2 = 0, columns_1 = 0, columns_2 = 0;
        for (;; ++n) {
            const int buf = n & 1, phase = (n >> 1) & 1;
            if (!open_step(n)) break;
            const Step &st = S.step[n % kSteps];
            const int subs = st.subs, first = st.first, last = st.last, rows = st.rows;
            const uint32_t shape = tc::mma_shape((rows + 15) & ~15, false, false);
            const int columns = F::kBoth ? 2 * ((rows + 7) & ~7) : (rows + 15) & ~15;  // of O
            close_step(n);
            if (first) wait(&S.q_full, items++ & 1);
            const int place = place_of_k(n), slot = place % slots;
            wait(&S.full[slot], (place / slots) & 1);
            if (n >= 2) wait(&S.s_free[buf], phase ^ 1);
            if (__any_sync(kAll, gave_up())) break;
            tc::fence_after();
            if (tc::elect_one()) {
#pragma unroll 1
                for (int u = 0; u < subs; ++u) {
#pragma unroll 1
                    for (int g = 0; g < kDigits; ++g)
#pragma unroll
                        for (int k = 0; k < D / 32; ++k)  // 32 channels further inside the swizzled rows
                            tc::mma_e4m3(tmem + buf * (kSub * N) + u * N, ring_k + ((slot * F::kSlot + u * kTile * D + k * 32) >> 4),
                                         q_desc + ((g * F::kQ + k * 32) >> 4), shape, g + k > 0);
                }
                tc::mma_commit(&S.s_full[buf]);
                tc::mma_commit(&S.empty[slot]);
                if (last) tc::mma_commit(&S.q_free);
            }
            __syncwarp();
            if (n >= 2) output_of(n - 2, subs_2, columns_2);
            subs_2 = subs_1, subs_1 = subs;
            columns_2 = columns_1, columns_1 = columns;
        }
        if (!__any_sync(kAll, gave_up())) {
            if (n >= 2) output_of(n - 2, subs_2, columns_2);
            if (n >= 1) output_of(n - 1, subs_1, columns_1);
        }
    } else if (warp == 14) {
// ---- the queries' digits: eight rows at a time, four lanes to a row ------------------
        constexpr int kPer = D / 4;  // channels per lane
        // scores of scale 0 are those of digits that are all 0
        const float sign = P.scale < 0.f ? -1.f : (P.scale > 0.f ? 1.f : 0.f), size = P.scale == 0.f ? 1.f : fabsf(P.scale);
        const int most = min(126, 126 + ilogbf(size));
        const int sub = lane >> 2, part_of_row = lane & 3;
        int items = 0;
        for (int it = 0;; ++it) {
            if (!open_step(it)) break;
            const Step &st = S.step[it % kSteps];
            if (st.first) {
                const int rows = st.rows, row0 = st.row0, token0 = st.token0, head0 = st.head * P.G, pos0 = st.pos0;
                uint4 x[kPer / 8];
                auto load = [&](int r) {
                    const int row = row0 + r;
                    const E *q = static_cast<const E *>(P.q) + (token0 + row / P.G) * P.q_stride +
                                 static_cast<int64_t>(head0 + row % P.G) * D + part_of_row * kPer;
#pragma unroll
                    for (int c = 0; c < kPer / 8; ++c)
                        x[c] = r < rows ? __ldg(reinterpret_cast<const uint4 *>(q) + c) : make_uint4(0, 0, 0, 0);
                };
                load(sub);
                if (items > 0) wait(&S.q_free, (items - 1) & 1);
#pragma unroll 1
                for (int r0 = 0; r0 < rows; r0 += 8) {
                    const int r = r0 + sub;
                    uint32_t two[kPer / 2];
#pragma unroll
                    for (int c = 0; c < kPer / 8; ++c) two[4 * c] = x[c].x, two[4 * c + 1] = x[c].y, two[4 * c + 2] = x[c].z, two[4 * c + 3] = x[c].w;
                    if (r0 + 8 < rows) load(r + 8);
                    float top = 0.f;
                    bool odd = false;
#pragma unroll
                    for (int c = 0; c < kPer; ++c) {
                        const float a = fabsf(wide(reinterpret_cast<const E *>(&two[c / 2])[c & 1]));
                        odd |= !(a <= 3.402823466e38f);
                        top = fmaxf(top, a);
                    }
                    top = fmaxf(top, __shfl_xor_sync(kAll, top, 1));
                    top = fmaxf(top, __shfl_xor_sync(kAll, top, 2));
                    odd = (__ballot_sync(kAll, odd) >> (lane & 28)) & 15;
                    // The largest is brought into [128, 256): k = 7 - its exponent.  Not so far that the factor of the
                    // scores, |scale| 2^-k, falls below the normal range: masked scores are -inf before it, and have to
                    // be so after it.
                    const int e = static_cast<int>(__float_as_uint(top) >> 23);
                    const int k = top == 0.f ? 0 : min(134 - e, most);
                    const float up = sign * __uint_as_float(static_cast<uint32_t>(127 + k) << 23);
#pragma unroll
                    for (int c0 = 0; c0 < kPer; c0 += 16) {  // one 16-byte chunk of each digit
                        uint32_t digit[kDigits][4];
#pragma unroll
                        for (int c = 0; c < 16; c += 2) {
                            const E *v = reinterpret_cast<const E *>(&two[(c0 + c) / 2]);
                            float a = wide(v[0]) * up, b = wide(v[1]) * up;
#pragma unroll
                            for (int g = 0; g < kDigits; ++g) {
                                const uint32_t d = e4m3x2(a, b);
                                const float2 f = floats_of_e4m3x2(d);
                                a -= f.x, b -= f.y;
                                digit[g][c / 4] = c % 4 == 0 ? d : digit[g][c / 4] | (d << 16);
                            }
                        }
#pragma unroll
                        for (int g = 0; g < kDigits; ++g)
                            *reinterpret_cast<uint4 *>(q_sh + g * F::kQ + tc::swizzled<D>(r, (part_of_row * kPer + c0) / 16)) =
                                make_uint4(digit[g][0], digit[g][1], digit[g][2], digit[g][3]);
                    }
                    if (part_of_row == 0) {
                        const bool there = r < rows;
                        const int pos = pos0 + (row0 + r) / P.G;
                        float f = size * __uint_as_float(static_cast<uint32_t>(127 - k) << 23);
                        if (odd) f = __int_as_float(0x7FC00000);
                        S.q_factor[items % kItems][r] = there ? f : 0.f;
                        S.row_last[items % kItems][r] = there ? pos : -1;
                    }
                }
                tc::fence_async_shared();
                __syncwarp();
                if (lane == 0) mbar_arrive(&S.q_full);
                ++items;
            }
            close_step(it);
        }
    } else {
        // ---- scout: items, pages and scales ahead of the others ---------------------------
        const int pages = F::kStep >> P.page_shift;  // of one step: 1 to 16
        const int at_once = 32 / pages;              // steps whose pages the lanes look up together
        const int my_step = lane / pages, my_page = lane % pages;
        Part part;
        int s = 0, items = 0;
        while (walk.next(P, part)) {
            if (__any_sync(kAll, gave_up())) break;
            const int low = part.pos0 + part.row0 / P.G, high = part.pos0 + (part.row0 + part.rows - 1) / P.G;
            const int common_to = low, common_from = P.window > 0 ? max(0, high + 1 - P.window) : 0;
            const int32_t *table = P.table + static_cast<int64_t>(part.b) * P.max_blocks;
            const int key0 = part.step * F::kStep;
            // page of this lane's place in the steps from t on; -1 for what is no page, less for what is no place
            constexpr int kNoPlace = -2;
            auto look_up = [&](int t) {
                const int j = key0 + (t + my_step) * F::kStep + (my_page << P.page_shift);
                const bool in = t + my_step < part.steps && j < part.stop && j + (1 << P.page_shift) > part.start;
                return in ? max(__ldg(table + (j >> P.page_shift)), -1) : kNoPlace;
            };
            int next = look_up(0);
            for (int t0 = 0; t0 < part.steps; t0 += at_once) {
                const int page = next;
                const bool there = page >= 0 && page < P.num_pages;
                float ks = 0.f, vs = 0.f;
                if (there) {
                    const int64_t block = static_cast<int64_t>(page) * P.Hkv + part.head;
                    ks = __ldg(P.ks + block);
                    vs = __ldg(P.vs + block);
                }
                if (page != kNoPlace && !there) report(P.dev_status, SSD_DEV_BAD_PAGE);
                if (t0 + at_once < part.steps) next = look_up(t0 + at_once);
                // Value scales are divided by a power of two above the step's largest, times 256: the weights'
                // digits start at e4m3's upper end.
                const bool finite = fabsf(vs) <= 3.402823466e38f;
                float top = finite ? fabsf(vs) : 0.f;
                for (int o = 1; o < pages; o <<= 1) top = fmaxf(top, __shfl_xor_sync(kAll, top, o));
                const uint32_t e = min(max(__float_as_uint(top) >> 23, 8u), 254u);
                const float f = finite ? vs * __uint_as_float((261u - e) << 23) : __int_as_float(0x7FC00000);
                const uint32_t there_all = __ballot_sync(kAll, there), odd_all = __ballot_sync(kAll, !finite);
                const uint32_t of_step = pages == 32 ? kAll : (1u << pages) - 1u;
                const int n = min(at_once, part.steps - t0);
                for (int i = 0; i < n; ++i, ++s) {
                    const int slot = s % kSteps;
                    if (s >= kSteps) wait(&S.step_free[slot], (s / kSteps - 1) & 1);
                    if (__any_sync(kAll, gave_up())) break;
                    Step &st = S.step[slot];
                    if (my_step == i) {
                        st.page[my_page] = page;
                        st.scale[my_page] = make_float2(ks, f);
                        if (my_page == 0) {
                            const int k0 = key0 + (t0 + i) * F::kStep;
                            const uint32_t mask = (there_all >> (i * pages)) & of_step;
                            st.live = 1;
                            st.first = t0 + i == 0;
                            st.last = t0 + i == part.steps - 1;
                            st.plain = mask == of_step && k0 >= common_from && k0 + F::kStep - 1 <= common_to;
                            st.odd = ((odd_all >> (i * pages)) & of_step) != 0;
                            st.key0 = k0;
                            st.subs = k0 + kTile < part.stop ? kSub : 1;
                            st.start = part.start, st.stop = part.stop;
                            st.common_from = common_from, st.common_to = common_to;
                            st.there = static_cast<int32_t>(mask);
                            st.item = items % kItems;
                            st.first_cta = part.first_cta, st.parts = part.parts;
                            st.seq = part.b, st.head = part.head, st.row0 = part.row0, st.rows = part.rows;
                            st.token0 = part.first, st.pos0 = part.pos0;
                            st.part_key0 = key0;
                            st.v_unit = __uint_as_float((e - 7u) << 23);
                        }
                    }
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&S.step_full[slot]);
                }
            }
            ++items;
        }
        // the end, once for each softmax group
        for (int i = 0; i < 2; ++i, ++s) {
            const int slot = s % kSteps;
            if (s >= kSteps) wait(&S.step_free[slot], (s / kSteps - 1) & 1);
            if (__any_sync(kAll, gave_up())) break;
            if (lane == 0) {
                S.step[slot].live = 0;
                mbar_arrive(&S.step_full[slot]);
            }
            __syncwarp();
        }
    }
    __syncwarp();
    if (tid == 0 && gave_up()) report(P.dev_status, SSD_DEV_TIMEOUT);
    tc::fence_before();
    __syncthreads();
    tc::fence_after();
    if (gave_up()) {
        // Some role left early, perhaps after the ones that issue copies and products had left: what they issued still
        // has to end before the CTA does.
        if (warp == 12) {
            const int highest = S.highest;
#pragma unroll 1
            for (int x = max(0, highest - slots + 1); x <= highest; ++x) drain_phase(&S.full[x % slots], (x / slots) & 1);
        }
        if (warp == 13) {
            if (tc::elect_one()) tc::mma_commit(&S.drained);
            __syncwarp();
            drain_phase(&S.drained, 0);
        }
    }
    if (warp == 13) tc::tmem_free(tmem, F::kColumns);
}

struct Device {
    int id = 0, sms = 0;
    int smem_cta = 0;
};
int device_limits(Device *d) {
    if (cudaGetDevice(&d->id) != cudaSuccess ||
        cudaDeviceGetAttribute(&d->sms, cudaDevAttrMultiProcessorCount, d->id) != cudaSuccess ||
        cudaDeviceGetAttribute(&d->smem_cta, cudaDevAttrMaxSharedMemoryPerBlockOptin, d->id) != cudaSuccess) {
        cudaGetLastError();
        return SSD_ERR_CUDA;
    }
    return SSD_OK;
}

template <class F>
int attend_launch(AttendParams P, const CUtensorMap &k_map, const CUtensorMap &v_map, const Device &dev, cudaStream_t stream) {
    auto *kernel = attend_kernel<F>;
    static_assert(kSlots<F> >= 4);
    const int dyn = kFixedBytes<F> + kSlots<F> * F::kSlot;
    if (dyn > dev.smem_cta) return SSD_ERR_UNSUPPORTED;
    static std::atomic<uint64_t> ready{0};  // devices on which this kernel may take that much
    const uint64_t bit = 1ull << (dev.id & 63);
    if (!(ready.load(std::memory_order_relaxed) & bit)) {
        if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, dyn) != cudaSuccess) {
            cudaGetLastError();
            return SSD_ERR_CUDA;
        }
        ready.fetch_or(bit, std::memory_order_relaxed);
    }
    P.rows_per_item = F::R;
    P.step_shift = log2_of(F::kStep);
    P.item_cost = F::kItemCost;
    P.inside = static_cast<int64_t>(P.max_new) * P.G <= F::R && P.B <= kSeqsInside;
    int ctas = dev.sms;
    if (ctas > kMaxCtas) ctas = kMaxCtas;
    if (!P.inside) {
        const int64_t most = static_cast<int64_t>(P.T) * P.G / F::R + P.B;
        if (most > kMaxPairs) return SSD_ERR_UNSUPPORTED;
        P.most_pairs = static_cast<int>(most);
        schedule_kernel<<<1, kScheduleThreads, 0, stream>>>(P, ctas);
        if (launched() != SSD_OK) return SSD_ERR_CUDA;
    }
    kernel<<<static_cast<unsigned>(ctas), kAttendThreads, static_cast<size_t>(dyn), stream>>>(P, k_map, v_map);
    if (launched() != SSD_OK) return SSD_ERR_CUDA;
    return SSD_OK;
}

// Rows of an item: 64 cost the outputs' registers and the weights' shared memory, so 32 where they hold every sequence.
template <class E, int D>
int attend_dispatch(const AttendParams &P, const CUtensorMap &k, const CUtensorMap &v, const Device &dev, cudaStream_t s) {
    if (static_cast<int64_t>(P.max_new) * P.G <= 32) return attend_launch<Form<E, D, 32>>(P, k, v, dev, s);
    return attend_launch<Form<E, D, 64>>(P, k, v, dev, s);
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
    const float scale = sm_scale * kLog2e;
    if (!(scale - scale == 0.f)) return SSD_ERR_INVALID_ARG;
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
    // Units of all items, which the schedule counts in 32 bits: steps of 128 or 256 keys, the last one begun, and up to
    // two for an item's start.
    const int64_t row_blocks = static_cast<int64_t>(T < 1 ? 1 : T) * (Hq / Hkv) / 8 + B;
    if (row_blocks * Hkv > 0x7FFFFFFF / (static_cast<int64_t>(max_blocks) * page_size / kTile + 3)) return SSD_ERR_UNSUPPORTED;
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
    P.scale = scale;
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
