// ssd_kv_attend_tree.cu -- attention of trees of new tokens over the paged e4m3 cache (sm_103a).
//
//   s_rj = sm_scale <q_r, k8_j> ks(page j),   out_r = sum_j softmax(s_r)_j v8_j vs(page j)
//
// over the positions before the tree and the nodes of a token's mask.  The rows r of one item are
// the tokens of a tree times the query heads that share one cache head, 256 of them at most: a tree
// has many rows where a decoded token has few, so the rows are the long side of both products.
//
// * S = Q K^T (128 rows x 128 keys) takes the keys as they lie in the cache.  A query row is scaled
//   by a power of two that brings its largest channel into [128, 256) and is the sum of two (bf16)
//   or three (fp16) e4m3 digits: exact down to 2^-9 or 2^-6 of that channel, off by 2^-17 of it at most.
// * A thread has a row of S: its maximum and sum cross no lanes, and a mask is 32 keys to a word.
// * The weights go back to TMEM as halves, over the scores they are made of, and are the A operand
//   of O = P V from there; V is turned into halves (exactly) once for all rows.  A weight is rounded
//   by 2^-11 of itself; it is held as 2^5 2^s vs / 2^m, with 2^m the largest 2^s vs of the keys that the row has
//   attended to, which may lag by 2^10: at most 2^15, and normal down to 2^-19 of the largest.  O stays in TMEM
//   from step to step, and is scaled there when m has to move on.  (Relative to a step's largest value scale, which a row need not attend to or which its largest
//   scores need not meet, weights lost bits that count.)
//
// Two streams of work pass through the tensor cores in turns, each with its S, O and four softmax
// warps: the two tiles of 128 rows of an item of more than 128, else every other step of its keys.
// While one stream's scores become weights, the other's products run.
//
// Roles of the warps: 0-7 softmax, scaling and output (a thread per row), 8-11 the queries' digits
// and V's halves, 12 TMA, 13 MMA, 14 the scout, which walks the items and looks up pages and scales.
//
// Work split.  All steps of all items form one line, which the CTAs (one to an SM) cut into equal
// stretches.  A CTA whose stretch ends inside an item leaves a partial result in the workspace, and
// the CTA that brings an item's last part joins them all.
//
// What bounds it (32/8 heads of 128, bf16, cold caches): 64 sequences of 37 nodes and 40 to 8191 keys
// 269 us, 578 MB of cache (85 us at the copy's rate) and two tiles for 148 rows; 4 of 9 nodes and 90001
// to 131072 keys 228 us (134 us of bytes); one of 37 nodes over 1074 keys 44 us.  DRAM is at 29% and
// 51%, the tensor pipe at 43%, issue at 40% and 45%: a step of two tiles would take the tensor cores
// 2144 clocks and takes some 3700, in which a stream's scores, weights and output follow one another
// through four softmax warps, and of an item's time as much as five steps is its start.  What binds the
// second case is not known: half the softmax chain (rows in two lanes, below) took 4 us off it.  The form
// that ssd_kv_attend has (keys as the long side) takes 170, 427 and 836 us for 64 sequences of 9, 32 and
// 64 tokens over these lengths, this one 163, 177 and 286; over the second case's very long sequences
// that form is the faster one with its 9 tokens (200 us).
//
// Clocks of one of a stream's passes, two tiles, when weights were relative to their step's value scales
// (267 us): 750 from the last weights to the next wait, 800 in it, 600 for the maximum, 1650 for the
// weights, 165 to store them; the MMA warp needs 1300 for its part.
//
// Tried and not faster (267, 222 and 44 us then): scores of 64 keys in two buffers a stream, so that a product runs beside the
// next pass's weights (323 us for the first case; 276 and 234 for the first two with both streams'
// products issued together, when the softmax warps bound every pass: a pass's fixed work comes twice);
// the next item's queries made during this one's steps (275; the same warps make V's halves); weights
// in loops of 32 keys (280) or with each load a loop ahead (299); all products of a pass from one
// instruction group (267); another slot for values in place of one for keys (269, and 349 in place of
// 302 in fp16); boxes fetched into L2 ahead of their copies (272); steps handed over two at a time
// (284); items of up to 64 rows with each row in two lanes, which take half the keys each (218 for
// the second case's 222, but 284 for the first, whose items are larger, by code alone, and 190 to 214
// for 165 with 64 trees of 9); whole rows in straight-line code, slower by the instruction caches.  A sum
// of the weights as rounded would cancel their common rounding, and lose keys of small value scales whose
// weights are none as halves.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <atomic>

#include "ssd_kv.h"
#include "ssd_tc.h"

namespace ssd {
namespace {

constexpr int kTile = 128;       // keys of a step, rows of a tile
constexpr int kMaxRows = 256;    // of an item
constexpr int kMaxHead = 128;
constexpr int kMaxCtas = 160;
constexpr int kInside = 256;        // (sequence, row block) pairs whose schedule every CTA makes itself
constexpr int kMaxPairs = 1 << 18;  // such pairs of a call
// What starting an item counts in the split, in steps.  With 4, 5, 6 and 9: the ragged batch of 37 nodes 265, 267, 269 and 278 us,
// of 32 nodes 190, 175, 173 and 175, of 64 289, 285, 288 and 298.
constexpr int kItemCost = 5;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kMost = 3.402823466e38f;
constexpr float kNothing = -3e38f;  // the maximum of a row that has attended to nothing
// Weights are 2^kUp times those relative to a row's largest, which may be passed by 2^kLag.
constexpr float kLag = 10.f, kUp = 15.f - kLag, kUnit = 32.f;  // (2^kUp)
// A pass takes the short form of the weights, relative to one number for their sum and for O, where value scales are from
// 2^-kMostUnit to 2^kMostUnit, so that the sum's terms down to 2^-(2 kMostUnit) are normal in fp32, and no score can
// be above 2^22.8: three roundings of 1/4 leave a weight below the largest half.  (A product of digits is at most 2^8 448
// kMostHead = 2^23.8, and mostly 2^8 less, which makes those roundings 2^-10.)  The long form's exponents are differences of
// scores, exact whatever their size, and a warp goes back to the short one while that is so to 2^-12.  It takes twice as long
// (the cases above 587, 472 and 63 us in place of 269, 228 and 44).
constexpr float kMostUnit = 50.f, kMostFactor = 0.5f, kMostScore = 8192.f;
// In the long form the sum is relative to the scores' maximum, and what the weights are relative to is not below 2^kLow
// (and kLag less) of that, so that it stays a normal number whatever the value scales.
constexpr float kLow = -109.f;

struct Workspace {
    float o[2 * kMaxCtas][kMaxHead][kMaxRows];
    float2 ml[2 * kMaxCtas][kMaxRows];
    int32_t arrived[kMaxCtas];  // parts of the item that starts in each CTA; left at 0
    int32_t pairs, seqs;        // of the schedule below, and sequences in it
    int32_t sums[kMaxPairs + 1];  // steps before each pair
    int32_t seq[kMaxPairs];
    int32_t row0[kMaxPairs];
    int32_t start[kMaxCtas + 1];  // pair in which each CTA's stretch starts
};

struct TreeParams {
    const void *q;
    int64_t q_stride;
    const uint8_t *v;
    const float *ks, *vs;
    int num_pages, page_shift, Hq, Hkv, G, g_shift;  // g_shift: of a G that is a power of two, else -1
    const int32_t *table;
    int max_blocks;
    const int32_t *cu, *kv_len, *mask;
    int words;  // of a token's mask
    int B, T, max_new;
    float scale;  // sm_scale * log2(e): scores are held in base 2
    int window;
    int inside;      // a sequence is a pair, and the schedule made by every CTA in shared memory
    int most_pairs;  // (sequence, row block) pairs that T tokens of B sequences can make
    int withheld;    // SSD_CHECK_..., 0: none
    void *out;
    Workspace *ws;
    int32_t *dev_status;
};

struct Seq {
    int first, n, pos0;  // first token, tokens served, position of the first
};
__device__ __forceinline__ Seq load_seq(const TreeParams &P, int b) {
    Seq s;
    s.first = min(max(P.cu[b], 0), P.T);
    const int n = min(max(P.cu[b + 1], s.first), P.T) - s.first;
    s.n = min(n, P.max_new);
    s.pos0 = max(P.kv_len[b], -(1 << 30)) - n;
    return s;
}

// The keys that any of rows [row0, row1) may attend to: [start, stop), in steps step0 .. step0 + steps.
struct Span {
    int start, stop, step0, steps;
};
__device__ __forceinline__ Span key_span(const TreeParams &P, const Seq &s, int row1) {
    const int high = s.pos0 + (row1 - 1) / P.G;
    Span k;
    k.start = P.window > 0 && s.pos0 > P.window ? s.pos0 - P.window : 0;
    k.stop = min(high + 1, P.max_blocks << P.page_shift);
    if (k.stop > k.start) {
        k.step0 = k.start / kTile;
        k.steps = (k.stop - 1) / kTile + 1 - k.step0;
    } else {  // nothing to attend to: one step without keys writes the zeros
        k.start = k.stop = k.step0 = 0;
        k.steps = 1;
    }
    return k;
}

// The node of a row, counted in its tree.
__device__ __forceinline__ int node_of(const TreeParams &P, int row) { return P.g_shift >= 0 ? row >> P.g_shift : row / P.G; }

__device__ __forceinline__ int first_unit(int64_t cta, int64_t units, int64_t ctas) {
    return static_cast<int>(cta * units / ctas);
}

// CTAs that share the line.  A stretch has some units at least: a part of few steps starts and ends like one of many, and
// all of an item's parts are read again by one CTA (one sequence of 37 nodes over 1074 keys: 48 us with 1 unit at least, 42
// with 4, 46 with 8; over 8000 keys 75, 70 and 65).
constexpr int kLeast = 6;
__device__ __forceinline__ int ctas_of(int most, int units) { return min(most, max(1, units / kLeast)) * (units > 0); }

// One item's part in a CTA's stretch.
struct Part {
    int b, head, row0, rows;
    int first, pos0;      // of the sequence
    int start, stop;      // keys that any row attends to
    int step, steps;      // this part's
    int first_cta, parts;  // CTAs that the item is cut over: first_cta and the parts - 1 after it
};

struct Walk {
    const int32_t *sums, *seq, *row0;  // (no seq: a pair is a sequence)
    int unit, end, pair;
    int units, ctas, cta;
    // A CTA's units are steps, after kItemCost units for the start of each item.
    __device__ __forceinline__ bool next(const TreeParams &P, Part &part) {
        for (;;) {
            if (unit >= end) return false;
            while (sums[pair + 1] <= unit) ++pair;
            const int base = sums[pair], all = (sums[pair + 1] - base) / P.Hkv;
            const int head = (unit - base) / all, done = (unit - base) - head * all - kItemCost;
            if (done < 0) {
                unit -= done;
                continue;
            }
            const int b = seq ? seq[pair] : pair;
            part.b = b;
            part.row0 = seq ? row0[pair] : 0;
            const Seq s = load_seq(P, b);
            part.first = s.first;
            part.pos0 = s.pos0;
            part.rows = min(kMaxRows, s.n * P.G - part.row0);
            const Span k = key_span(P, s, part.row0 + part.rows);
            part.start = k.start, part.stop = k.stop;
            part.head = head;
            part.step = k.step0 + done;
            part.steps = min(k.steps - done, end - unit);
            part.first_cta = cta, part.parts = 1;
            if (part.steps < k.steps) {
                const int64_t item = static_cast<int64_t>(base) + static_cast<int64_t>(head) * all;
                part.first_cta = static_cast<int>(((item + kItemCost + 1) * ctas - 1) / units);
                part.parts = static_cast<int>(((item + all) * ctas - 1) / units) - part.first_cta + 1;
            }
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

// The schedule: the (sequence, row block) pairs, and the units before each in sums [pairs + 1], of which the total is
// returned.  seqs: the sequences() in it.  blocks [B + 1] is for the block's own use.
template <int kN>
__device__ __forceinline__ int make_schedule(const TreeParams &P, int32_t *blocks, int32_t *sums, int32_t *seq, int32_t *row0,
                                             int *red, int &pairs, int &seqs) {
    const int tid = threadIdx.x;
    int carry = 0;
    if (tid == 0) blocks[0] = 0;
    for (seqs = P.B;; seqs = sequences<kN>(P.cu, P.B, red)) {  // (counted once where cu_new does not fall)
        bool falls = false;
        carry = 0;
        for (int base = 0; base < seqs; base += kN) {
            const int b = base + tid;
            int v = 0;
            if (b < seqs) v = (load_seq(P, b).n * P.G + kMaxRows - 1) / kMaxRows, falls |= P.cu[b + 1] < P.cu[b];
            const int sum = block_sums<kN>(v, carry, red);
            if (b < seqs) blocks[b + 1] = sum;
        }
        if (!__syncthreads_or(falls)) break;
    }
    pairs = min(carry, P.most_pairs);  // (what the tokens of that many sequences can make)
    carry = 0;
    if (tid == 0) sums[0] = 0;
    for (int base = 0; base < pairs; base += kN) {
        const int p = base + tid;
        int v = 0;
        if (p < pairs) {
            const int b = last_not_above(blocks, seqs, p);
            const int first = (p - blocks[b]) * kMaxRows;
            const Seq s = load_seq(P, b);
            v = (key_span(P, s, min(first + kMaxRows, s.n * P.G)).steps + kItemCost) * P.Hkv;
            seq[p] = b;
            row0[p] = first;
        }
        const int sum = block_sums<kN>(v, carry, red);
        if (p < pairs) sums[p + 1] = sum;
    }
    __syncthreads();
    return carry;
}

// The schedule of a call of more than kInside pairs: one CTA.
constexpr int kScheduleThreads = 1024;
__global__ void __launch_bounds__(kScheduleThreads) schedule_kernel(const __grid_constant__ TreeParams P, int ctas) {
    __shared__ int32_t blocks[SSD_KV_MAX_B + 1];
    __shared__ int red[kScheduleThreads / 32];
    Workspace &W = *P.ws;
    int pairs, seqs;
    const int units = make_schedule<kScheduleThreads>(P, blocks, W.sums, W.seq, W.row0, red, pairs, seqs), used = ctas_of(ctas, units);
    if (threadIdx.x == 0) W.pairs = pairs, W.seqs = seqs;
    for (int c = threadIdx.x; c < used; c += kScheduleThreads)
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
__device__ __forceinline__ uint32_t two_of(__nv_bfloat16, float a, float b) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&v);
}
__device__ __forceinline__ uint32_t two_of(__half, float a, float b) {
    const __half2 v = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&v);
}
// Two halves as e4m3, the low one in the low byte; rounding and range as e4m3x2.
__device__ __forceinline__ uint32_t e4m3x2_of_halves(__half2 v) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(r) : "r"(*reinterpret_cast<const uint32_t *>(&v)));
    return r;
}
// Two fp32 values in one register pair, and their arithmetic in one instruction.
__device__ __forceinline__ uint64_t pack2(float a, float b) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ void unpack2(uint64_t v, float &a, float &b) { asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v)); }
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
// The largest, NaN left out.
__device__ __forceinline__ float max3(float a, float b, float c) {
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}
// Of numbers below the normal range, too.
__device__ __forceinline__ float lg2_of_any(float x) {
    float r;
    asm("lg2.approx.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
__device__ __forceinline__ void prefetch(const void *p) { asm volatile("prefetch.global.L2 [%0];" ::"l"(p)); }
// 2^(e - 127)
__device__ __forceinline__ float power(int e) { return __uint_as_float(static_cast<uint32_t>(e) << 23); }

constexpr int kTreeWarps = 16;  // softmax 2 x 4, digits and halves 4, TMA, MMA, scout, one that only makes up the last four
constexpr int kTreeThreads = 32 * kTreeWarps;
constexpr int kRegisters = 128, kSoftmaxRegisters = 168, kOtherRegisters = 88;  // of a thread: at launch, and then
static_assert(kSoftmaxRegisters + kOtherRegisters <= 2 * kRegisters && kRegisters * kTreeThreads <= 65536);
constexpr int kSteps = 8;   // steps that the scout may be ahead
constexpr int kItems = 4;   // items whose row data may be in use at once
constexpr int kGroups = 8;  // of 16 keys, the smallest page, in a step
constexpr int kConsumers = 8 + 4 + 2;  // warps that read a step

template <class E_, int kD_>
struct Form {
    using E = E_;
    static constexpr int D = kD_;
    static constexpr int kDigits = __is_same(E, __half) ? 3 : 2;
    static constexpr int kSlot = kTile * D;       // bytes of a step's keys, values, or one digit of a tile of queries
    static constexpr int kHalves = 2 * kSlot;     // of a step's values as halves
    static constexpr int kKeys = D == 64 ? 6 : (kDigits == 3 ? 2 : 3);  // slots of the rings
    static constexpr int kValues = D == 64 ? 4 : (kDigits == 3 ? 1 : 2);
    static constexpr int kBytes = 1024 + 2 * kDigits * kSlot + 2 * kHalves + (kKeys + kValues) * kSlot;
    static constexpr int kO = 256;  // TMEM column of the first output; the scores' are 0 and 128
};

// One step of a CTA's stretch: up to kTile keys of one item.
constexpr int kLive = 1;       // 0: the stretch has ended
constexpr int kPair = 2;       // two tiles of rows: both streams take part in every step
constexpr int kBegins = 4, kEnds = 8;   // first, last step of its part
constexpr int kFirst = 16, kLast = 32;  // its passes are the part's first, last of their streams
constexpr int kWhole = 64;     // every row attends to every key, and every page is there
constexpr int kOrdinary = 128;  // the pages' scales are ordinary numbers
constexpr int kStream = 256;   // stream of the step's first pass
constexpr int kSingle = 512;   // the part is this step alone
struct Step {
    int32_t flags;
    int32_t key0;
    int32_t start, stop;  // keys that some row attends to
    int32_t common_from, common_to;  // ... and that every row does
    int32_t there;        // bit g: group g's page is there
    int32_t item;         // of kItems
    int32_t first_cta, parts;  // of the item
    int32_t seq, head, row0, rows, token0, pos0;
    int32_t part_key0;    // first key of the part
    float k_most;         // the largest scale of its keys, where all are ordinary
    int32_t page[kGroups];
    // of the keys, and of the values (NaN if not finite); the logarithm (base 2) of the latter's size, and its reciprocal
    alignas(16) float4 scale[kGroups];
};

template <class F>
struct Shared {
    uint64_t k_full[F::kKeys], k_empty[F::kKeys], v_full[F::kValues], v_empty[F::kValues];
    uint64_t step_full[kSteps], step_free[kSteps];
    uint64_t h_full[2], h_free[2];  // V's halves
    uint64_t s_full[2], p_full[2], o_full[2], o_free[2], q_full, q_free, meet, drained;
    Step step[kSteps];
    float q_factor[kItems][kMaxRows];
    float2 stat[2][2][kTile];  // maxima and sums of the streams, of every other item
    float unit[2][2][kTile];   // what their weights are relative to
    uint32_t tmem;
    int nan_met[kItems];  // NaN among an item's values that only some rows attend to
    int gave_up;
    int k_issued, v_issued;  // copies
    int last_part;
    int red[kTreeWarps];
};

// A whole warp waits, and its lanes get the same answer: loops and branches that the compiler takes for divergent cost
// this kernel more than anything else in a wait (one lane that waits for all: 411 us in place of 288).  Waits are
// bounded by a number of polls (each suspends the warp for 4 us at most: 4 s in all, far more than any step takes).
// When one runs out, `gave_up` is set and every role leaves its loop without waiting for the others; no role meets
// another at a barrier that is not waited for in this way.
constexpr int kPolls = 1 << 20, kPollsChecked = 1 << 12;
template <int kLimit>
__device__ __forceinline__ bool wait_phase(uint64_t *bar, uint32_t parity, volatile int *gave_up) {
    for (int polls = 0; !__all_sync(0xFFFFFFFFu, mbar_try_wait(bar, parity)); ++polls) {
        if (__any_sync(0xFFFFFFFFu, *gave_up) || polls == kLimit) {
            *gave_up = 1;
            return false;
        }
    }
    return true;
}
// The same for what has to end whether or not a wait ran out.
template <int kLimit>
__device__ __forceinline__ void drain_phase(uint64_t *bar, uint32_t parity) {
    for (int i = 0; i < kLimit && !mbar_try_wait(bar, parity); ++i) {
    }
}

// What a row attends to: every position from `from` up to pos0, and the nodes from `node_from` to `node` of its mask.
struct Row {
    const int32_t *mask;  // NULL for a row that is not there
    int node, node_from, from;
};
__device__ __forceinline__ Row load_row(const TreeParams &P, int token0, int pos0, int row, bool there) {
    Row r{};
    if (!there) {
        r.node = -1, r.from = 0x7FFFFFFF;
        return r;
    }
    r.node = row / P.G;
    r.mask = P.mask + static_cast<int64_t>(token0 + r.node) * P.words;
    if (P.window > 0) {
        // the last `window` keys: nodes from the highest one down, then positions before the tree
        int left = P.window;
        for (int w = r.node >> 5; w >= 0 && left > 0; --w) {
            uint32_t bits = static_cast<uint32_t>(__ldg(r.mask + w));
            if (w == r.node >> 5) bits &= 0xFFFFFFFFu >> (31 - (r.node & 31));
            const int n = __popc(bits);
            if (n > left) {
                for (int drop = n - left; drop > 0; --drop) bits &= bits - 1;
                r.node_from = 32 * w + __ffs(bits) - 1;
            }
            left -= min(n, left);
            if (left == 0 && n > 0 && r.node_from == 0) r.node_from = 32 * w + __ffs(bits) - 1;
        }
        r.from = left == 0 ? 0x7FFFFFFF : (pos0 > left ? pos0 - left : 0);
    }
    return r;
}
// Bits of the kTile keys from `key` on that a row attends to, whatever pages are there.
__device__ __forceinline__ void row_keys(const TreeParams &P, const Row &r, int pos0, int key, uint32_t (&bits)[4]) {
    const int node0 = key - pos0, w0 = node0 >> 5, shift = node0 & 31;
    uint32_t word[5];
#pragma unroll
    for (int i = 0; i < 5; ++i) {
        const int w = w0 + i;
        word[i] = w >= 0 && w <= r.node >> 5 ? static_cast<uint32_t>(__ldg(r.mask + w)) : 0u;  // (a row that is not there has node -1)
    }
#pragma unroll
    for (int c = 0; c < 4; ++c) {
        const int first = node0 + 32 * c;
        uint32_t b = __funnelshift_r(word[c], word[c + 1], shift);
        if (first > r.node || first + 31 < r.node_from) b = 0;
        const uint32_t last = static_cast<uint32_t>(r.node) - static_cast<uint32_t>(first);
        const uint32_t low = static_cast<uint32_t>(r.node_from) - static_cast<uint32_t>(first);
        if (last < 31u) b &= (2u << last) - 1u;
        if (low < 32u) b &= 0xFFFFFFFFu << low;
        // positions before the tree
        const int to = min(-first, 32), from = r.from - (key + 32 * c);
        if (to > 0 && from < to) b |= (0xFFFFFFFFu >> (32 - to)) & (from > 0 ? 0xFFFFFFFFu << from : 0xFFFFFFFFu);
        bits[c] = b;
    }
}

// A row of O times f.
template <class F>
__device__ __forceinline__ void scale_output(uint32_t o_at, float f) {
#pragma unroll 1
    for (int c = 0; c < F::D; c += 16) {
        uint32_t o[16];
        tc::tmem_load(o, o_at + c);
        tc::tmem_wait_load(o);
#pragma unroll
        for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * f);
        tc::tmem_store(o_at + c, o);
    }
}

// The long form of a step's weights; out of the kernel's loop, whose code it would lengthen (273, 226 and 46 us for the cases
// above).
struct State {
    float m, l, u;
};
template <class F>
__device__ __noinline__ State long_weights(const Step &st, State row, float qf, bool first, uint32_t sees_0, uint32_t sees_1, uint32_t sees_2,
                                           uint32_t sees_3, uint32_t s_at, uint32_t o_at) {
    constexpr uint32_t kAll = 0xFFFFFFFFu;
    const uint32_t sees[4] = {sees_0, sees_1, sees_2, sees_3};
    float m = row.m, l = row.l, u = row.u;
    float x[16], to = m, largest = -INFINITY;
#pragma unroll 1
    for (int c = 0; c < 2 * kGroups; ++c) {  // the largest score and weight, then the weights
        const int g = c & (kGroups - 1);
        const float4 sc = st.scale[g];
        const uint32_t bits = (g < 4 ? (g < 2 ? sees[0] : sees[1]) : (g < 6 ? sees[2] : sees[3])) >> (16 * (g & 1));
        const float f = sc.x * qf;
        if (c == kGroups) {
            largest = fmaxf(largest, kLow);
            if (first) {
                m = to, u = largest;
            } else {
                const float up = to - m;
                l *= ex2(-up);
                m = to, u -= up;
                const bool move = largest > u + kLag;
                if (__any_sync(kAll, move)) {
                    scale_output<F>(o_at, move ? ex2(u - largest) : 1.f);
                    if (move) u = largest;
                }
            }
        }
        tc::tmem_load(x, s_at + 16 * g);
        tc::tmem_wait_load(x);
#pragma unroll
        for (int i = 0; i < 16; ++i) x[i] = (bits >> i) & 1 ? x[i] * f : -INFINITY;
        if (c < kGroups) {
            float top = x[0];
#pragma unroll
            for (int i = 1; i < 16; ++i) top = fmaxf(top, x[i]);
            const float before = to;
            to = fmaxf(to, top);
            largest = fmaxf(largest - (to - before), (top - to) + sc.z);
            continue;
        }
        const float e = sc.z + (kUp - u);
        uint32_t w[8];
        float sum = 0.f;
#pragma unroll
        for (int i = 0; i < 16; i += 2) {
            float y = x[i] - m, z = x[i + 1] - m;
            sum += ex2(y) + ex2(z);
            // (not 0 times a scale that is not finite, of keys that the row does not attend to)
            y = (bits >> i) & 1 ? copysignf(ex2(y + e), sc.y) : 0.f, z = (bits >> i) & 2 ? copysignf(ex2(z + e), sc.y) : 0.f;
            w[i / 2] = two_of(__half(), y, z);
        }
        l += sum;
        tc::tmem_store(s_at + 8 * g, w);
    }
    return {m, l, u};
}

// kOwn: a schedule of several row blocks to a sequence is made by every CTA (as a branch it cost the others 1%).
// kChecked: the form of ssd_check_tree_timeout: in each CTA the third step's signal of role P.withheld is left out, so that
// the waits for it run out, after kPollsChecked polls.
template <class F, bool kOwn, bool kChecked = false>
__global__ void __launch_bounds__(kTreeThreads, 1)
    tree_kernel(const __grid_constant__ TreeParams P, const __grid_constant__ CUtensorMap k_map,
                const __grid_constant__ CUtensorMap v_map) {
    using E = typename F::E;
    constexpr int D = F::D, kDigits = F::kDigits;
    constexpr uint32_t kAll = 0xFFFFFFFFu;
    extern __shared__ uint8_t raw[];
    uint8_t *base = raw + ((1024 - (smem_addr(raw) & 1023)) & 1023);
    uint8_t *q_sh = base;                              // [tile][digit]
    uint8_t *h_sh = q_sh + 2 * kDigits * F::kSlot;     // V's halves, two steps
    uint8_t *k_sh = h_sh + 2 * F::kHalves;
    uint8_t *v_sh = k_sh + F::kKeys * F::kSlot;
    Shared<F> &S = *reinterpret_cast<Shared<F> *>(v_sh + F::kValues * F::kSlot);
    int32_t *sums_sh = reinterpret_cast<int32_t *>(&S + 1);
    const int tid = threadIdx.x, lane = tid & 31;
    const int warp = __shfl_sync(kAll, tid >> 5, 0);
    const int cta = blockIdx.x;

    if (tid == 0) tc::prefetch_map(&k_map), tc::prefetch_map(&v_map);
    // ---- schedule -------------------------------------------------------------------
    Walk walk;
    int pairs, seqs = P.B;
    if constexpr (kOwn) {
        int32_t *blocks = sums_sh + kInside + 1, *seq = blocks + kInside + 1, *row0 = seq + kInside;
        walk.units = make_schedule<kTreeThreads>(P, blocks, sums_sh, seq, row0, S.red, pairs, seqs);
        walk.sums = sums_sh, walk.seq = seq, walk.row0 = row0;
    } else if (P.inside) {
        int carry = 0;
        if (tid == 0) sums_sh[0] = 0;
        for (;; seqs = sequences<kTreeThreads>(P.cu, P.B, S.red)) {
            static_assert(kInside <= kTreeThreads);
            int v = 0;
            bool falls = false;
            if (tid < seqs) {
                const Seq s = load_seq(P, tid);
                if (s.n > 0) v = (key_span(P, s, s.n * P.G).steps + kItemCost) * P.Hkv;
                falls = P.cu[tid + 1] < P.cu[tid];
            }
            carry = 0;
            const int sum = block_sums<kTreeThreads>(v, carry, S.red);
            if (tid < seqs) sums_sh[tid + 1] = sum;
            if (!__syncthreads_or(falls)) break;
        }
        pairs = seqs;
        walk.sums = sums_sh;
        walk.units = carry;
        walk.seq = walk.row0 = nullptr;
    } else {
        walk.sums = P.ws->sums, walk.seq = P.ws->seq, walk.row0 = P.ws->row0;
        pairs = P.ws->pairs, seqs = P.ws->seqs;
        walk.units = P.ws->sums[pairs];
    }
    walk.ctas = ctas_of(static_cast<int>(gridDim.x), walk.units);
    walk.cta = cta;
    const bool busy = cta < walk.ctas;
    walk.unit = busy ? first_unit(cta, walk.units, walk.ctas) : 0;
    walk.end = busy ? first_unit(cta + 1, walk.units, walk.ctas) : 0;
    walk.pair = !busy ? 0 : (kOwn || P.inside ? last_not_above(sums_sh, pairs, walk.unit) : P.ws->start[cta]);

    // Tokens that no item serves get zeros: those behind the last sequence's, and those beyond max_new.
    {
        const int64_t width = static_cast<int64_t>(P.Hq) * D;
        E *out = static_cast<E *>(P.out);
        const int64_t stride = static_cast<int64_t>(gridDim.x) * kTreeThreads;
        const int served = min(max(P.cu[seqs], 0), P.T);
        for (int64_t i = served * width + static_cast<int64_t>(cta) * kTreeThreads + tid; i < P.T * width; i += stride)
            out[i] = narrow<E>(0.f);
        for (int b = cta; b < P.B; b += gridDim.x) {
            const int first = P.cu[b], next = P.cu[b + 1], keys = P.kv_len[b];
            const int from = min(max(first, 0), P.T), to = min(max(next, from), P.T);
            // a length counts where tokens are there to attend over it
            const bool fits = first >= 0 && next >= first && next <= P.T &&
                              (to == from || (keys >= 0 && keys <= P.max_blocks << P.page_shift));
            if (tid == 0 && (!fits || to - from > P.max_new)) report(P.dev_status, SSD_DEV_BAD_LENGTH);
            if (b >= seqs) continue;
            for (int64_t i = (from + P.max_new) * width + tid; i < to * width; i += kTreeThreads) out[i] = narrow<E>(0.f);
        }
    }

    if (tid == 0) {
        for (int i = 0; i < F::kKeys; ++i) mbar_init(&S.k_full[i], 1), mbar_init(&S.k_empty[i], 4);
        for (int i = 0; i < F::kValues; ++i) mbar_init(&S.v_full[i], 1), mbar_init(&S.v_empty[i], 4);
        for (int i = 0; i < kSteps; ++i) mbar_init(&S.step_full[i], 1), mbar_init(&S.step_free[i], kConsumers);
        for (int i = 0; i < 2; ++i) {
            mbar_init(&S.h_full[i], 4);
            mbar_init(&S.h_free[i], 1);
            mbar_init(&S.s_full[i], 1);
            mbar_init(&S.p_full[i], 4);
            mbar_init(&S.o_full[i], 1);
            mbar_init(&S.o_free[i], 8);
        }
        mbar_init(&S.q_full, 4);
        mbar_init(&S.q_free, 1);
        mbar_init(&S.meet, 8);
        mbar_init(&S.drained, 1);
        for (int i = 0; i < kItems; ++i) S.nan_met[i] = 0;
        S.gave_up = 0;
        S.k_issued = S.v_issued = 0;
        fence_mbar_init();
    }
    if (busy && warp == 13) tc::tmem_alloc(&S.tmem, 512);
    tc::fence_before();
    __syncthreads();
    tc::fence_after();
    if (!busy) return;
    const uint32_t tmem = S.tmem;
    // a softmax thread holds half a row of scores, and their weights
    if (warp < 8)
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftmaxRegisters));
    else
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegisters));

    constexpr int kWait = kChecked ? kPollsChecked : kPolls;
    auto wait = [&](uint64_t *bar, int parity) { return wait_phase<kWait>(bar, static_cast<uint32_t>(parity), &S.gave_up); };
    auto withheld = [&](int role, int step) { return kChecked && P.withheld == role && step == 2; };
    auto gave_up = [&] { return *static_cast<volatile int *>(&S.gave_up) != 0; };
    // The flags of step s, for all lanes of a warp; 0 at the end, or where a wait ran out.
    auto open_step = [&](int s) {
        const bool there = wait(&S.step_full[s % kSteps], (s / kSteps) & 1);
        const int flags = S.step[s % kSteps].flags;
        return static_cast<int>(__reduce_or_sync(kAll, there ? static_cast<uint32_t>(flags) : 0u));
    };
    auto arrive = [&](uint64_t *bar) {
        __syncwarp();
        tc::warp_arrive(bar);
    };

    if (warp < 8) {
        // ---- softmax: one row per thread -------------------------------------------------
        const int group = warp >> 2, quad = warp & 3, at_row = tid & 127;
        const uint32_t lanes = static_cast<uint32_t>(quad) << 21;
        const uint32_t s_at = tmem + group * kTile + lanes, o_at = tmem + F::kO + group * D + lanes;
        int ended[2] = {0, 0}, meets = 0, shared = 0;  // items whose output a stream has finished; meetings of the two groups; items of one tile
        Row row{};
        // what the row's sum is relative to, the sum, and what the weights in O are relative to that (0 but in the long form)
        float m = 0.f, l = 0.f, u = 0.f, qf = 0.f;
        int passes = 0, r = 0, k_slot = 0;  // of the stream; this thread's row of the item; of the step's keys
        bool any = false, some = false;  // the warp has rows; the row has attended to a key
        bool far = false;  // a row of the warp is one that only the long form serves
        for (int it = 0;; ++it) {
            const int flags = open_step(it);
            if (!(flags & kLive)) break;
            const Step &st = S.step[it % kSteps];
            const bool pair = flags & kPair, other = ((flags & kStream) != 0) != (group != 0);  // the step's first pass is not this stream's
            if (flags & kBegins) {
                const int rows = st.rows;
                r = at_row + (pair && other ? kTile : 0);
                any = __any_sync(kAll, r < rows);
                row = load_row(P, st.token0, st.pos0, st.row0 + r, r < rows);
                m = kNothing, l = 0.f, u = 0.f, qf = 0.f, some = false, far = false;
            }
            if (pair || !other) {
                const bool first = flags & kFirst;
                uint32_t sees[4] = {kAll, kAll, kAll, kAll};
                if (any && !(flags & kWhole)) {  // (while the scores are made)
                    row_keys(P, row, st.pos0, st.key0, sees);
                    const uint32_t there = st.there;
#pragma unroll
                    for (int c = 0; c < 4; ++c) sees[c] &= ((there >> (2 * c)) & 1 ? 0xFFFFu : 0u) | ((there >> (2 * c)) & 2 ? 0xFFFF0000u : 0u);
                }
                // (qf is 0 before the first scores, whose factors are there with them)
                bool ordinary = (flags & kOrdinary) && !far && !__any_sync(kAll, qf * st.k_most > kMostFactor);
                if (!wait(&S.s_full[group], passes++ & 1)) break;
                tc::fence_after();
                if (pair == other) tc::warp_arrive(&S.k_empty[k_slot]);  // the step's last scores are there
                if (any) {
                    if (first) {
                        qf = r < st.rows ? S.q_factor[st.item][r] : 0.f;
                        ordinary = ordinary && !__any_sync(kAll, qf * st.k_most > kMostFactor);
                    }
                    // Of the scores.  Not 0 where it is small, so that a masked one stays below all others.
                    auto factor = [&](float ks) {
                        const float f = ks * qf;
                        return f <= 1.2e-38f ? 1.2e-38f : f;
                    };
                    some |= (sees[0] | sees[1] | sees[2] | sees[3]) != 0;
                    // Loops of few instructions: straight-line code for a whole row of scores passes through the instruction
                    // caches each time, and the other roles' code with it.
                    if (ordinary) {
                        float x[4][16], top = -INFINITY;
                        auto fetch = [&](int c) {
#pragma unroll
                            for (int h = 0; h < 4; ++h) tc::tmem_load(x[h], s_at + 64 * c + 16 * h);
                        };
                        auto arrived = [&](int c) {
                            tc::tmem_wait_load(x);
                            if (!(flags & kWhole)) {
                                const uint32_t lo = c ? sees[2] : sees[0], hi = c ? sees[3] : sees[1];
#pragma unroll
                                for (int h = 0; h < 4; ++h)
#pragma unroll
                                    for (int i = 0; i < 16; ++i)
                                        x[h][i] = (h < 2 ? lo : hi) & (1u << (16 * (h & 1) + i)) ? x[h][i] : -INFINITY;
                            }
                        };
                        fetch(0);
#pragma unroll 1
                        for (int c = 0; c < 2; ++c) {
                            float f[4], e[4];
#pragma unroll
                            for (int h = 0; h < 4; ++h) f[h] = factor(st.scale[4 * c + h].x), e[h] = st.scale[4 * c + h].z;
                            arrived(c);
                            float w[4];
#pragma unroll
                            for (int h = 0; h < 4; ++h) {
                                float t = max3(x[h][0], x[h][1], x[h][2]), v = max3(x[h][3], x[h][4], x[h][5]);
#pragma unroll
                                for (int i = 6; i < 14; i += 4) t = max3(t, x[h][i], x[h][i + 1]), v = max3(v, x[h][i + 2], x[h][i + 3]);
                                w[h] = fmaf(max3(fmaxf(t, v), x[h][14], x[h][15]), f[h], e[h]);
                            }
                            fetch(1 - c);
                            top = fmaxf(top, fmaxf(fmaxf(w[0], w[1]), fmaxf(w[2], w[3])));
                        }
                        // What the weights are relative to moves on where it is passed by 2^kLag, and O and the sum follow.
                        if (first) {
                            m = fmaxf(top, kNothing);
                        } else if (const bool move = top > m + kLag; __any_sync(kAll, move)) {
                            const float to = move ? top : m, by = ex2(m - to);
                            l *= by;
                            m = to;
                            scale_output<F>(o_at, by);
                        }
                        // 2^s vs / 2^m is one power here, and the sum over 16 keys is divided by vs.
                        const float unit = kUp - m;
                        float sums = 0.f;
                        // (the first 64 scores' weights lie over themselves: the second 64 follow them)
#pragma unroll 1
                        for (int c = 0; c < 2; ++c) {
                            arrived(c);
                            uint32_t w[4][8];
#pragma unroll
                            for (int h = 0; h < 4; ++h) {
                                const float4 sc = st.scale[4 * c + h];
                                const float f = factor(sc.x), e = sc.z + unit;
                                const uint64_t f2 = pack2(f, f), e2 = pack2(e, e);
                                uint64_t s2 = 0;
#pragma unroll
                                for (int i = 0; i < 16; i += 2) {
                                    float y, z;
                                    unpack2(fma2(pack2(x[h][i], x[h][i + 1]), f2, e2), y, z);
                                    y = ex2(y), z = ex2(z);
                                    s2 = add2(s2, pack2(y, z));
                                    w[h][i / 2] = two_of(__half(), y, z);
                                }
                                float y, z;
                                unpack2(s2, y, z);
                                sums = fmaf(y + z, sc.w, sums);
                            }
                            if (c == 0) fetch(1);
#pragma unroll
                            for (int h = 0; h < 4; ++h) tc::tmem_store(s_at + 32 * c + 8 * h, w[h]);
                        }
                        l = fmaf(sums, 1.f / kUnit, l);
                    } else {
                        const State now = long_weights<F>(st, {m, l, u}, qf, first, sees[0], sees[1], sees[2], sees[3], s_at, o_at);
                        m = now.m, l = now.l, u = now.u;
                        // back to one number for both, where that is in range
                        const bool none = m == kNothing;
                        far = __any_sync(kAll, !none && (fabsf(u) > kMostUnit || fabsf(m) > kMostScore));
                        if (!far) {
                            if (!none) m += u, l *= ex2(-u);
                            u = 0.f;
                        }
                    }
                    tc::tmem_wait_store();
                    tc::fence_before();
                }
                if (withheld(SSD_CHECK_WEIGHTS, it) && quad == 0)
                    __syncwarp();
                else
                    arrive(&S.p_full[group]);
            }
            if (flags & kEnds) {
                // ---- the item's output, or this part's share of it ----
                const int took = pair || !(flags & kSingle) ? 3 : (flags & kStream ? 2 : 1);
                const int ch0 = pair ? 0 : group * (D / 2), chs = pair ? D : D / 2;  // the two groups share a single tile
                if (!some) m = kNothing, l = 0.f, u = 0.f;
                float mul_0 = 0.f, mul_1 = 0.f, total = l, top = m;
                bool fine = true;
                if (pair) {
                    (group ? mul_1 : mul_0) = ex2(u - kUp);
                    fine = wait(&S.o_full[group], ended[group] & 1);
                } else {
                    // (the other group may still read what the item before left)
                    const int buf = shared++ & 1;
                    S.stat[buf][group][at_row] = make_float2(m, l);
                    S.unit[buf][group][at_row] = u;
                    arrive(&S.meet);
                    fine = wait(&S.meet, meets++ & 1);
                    float2 both[2];
#pragma unroll
                    for (int g = 0; g < 2; ++g) both[g] = (took >> g) & 1 ? S.stat[buf][g][at_row] : make_float2(kNothing, 0.f);
                    top = fmaxf(both[0].x, both[1].x);
                    total = 0.f;
#pragma unroll
                    for (int g = 0; g < 2; ++g) {
                        if (!((took >> g) & 1)) continue;
                        const float down = both[g].x - top;
                        total = fmaf(both[g].y, ex2(down), total);
                        (g ? mul_1 : mul_0) = ex2(down + (S.unit[buf][g][at_row] - kUp));
                        fine &= wait(&S.o_full[g], ended[g] & 1);
                    }
                }
                if (__any_sync(kAll, !fine)) break;
                tc::fence_after();
                const int parts = st.parts, first_cta = st.first_cta;
                const bool mine = r < st.rows, nothing = top == kNothing;
                const bool use_0 = pair ? group == 0 : (took & 1) != 0, use_1 = pair ? group == 1 : (took & 2) != 0;
                auto slot_of = [&](int c) { return 2 * c + (c == first_cta ? 1 : 0); };
                const int node = (st.row0 + r) / P.G, head = st.head * P.G + (st.row0 + r) - node * P.G;
                E *out = static_cast<E *>(P.out) + (static_cast<int64_t>(st.token0 + node) * P.Hq + head) * D;
                Workspace &W = *P.ws;
                const int slot = slot_of(cta);
                auto store = [&](int ch, const float *x, float f) {  // 16 channels
                    uint32_t w[8];
#pragma unroll
                    for (int i = 0; i < 16; i += 2) w[i / 2] = two_of(E(), x[i] * f, x[i + 1] * f);
                    uint4 *at = reinterpret_cast<uint4 *>(out + ch);
                    at[0] = make_uint4(w[0], w[1], w[2], w[3]), at[1] = make_uint4(w[4], w[5], w[6], w[7]);
                };
                if (any) {
                    const float f = parts > 1 ? 1.f : (total == 0.f ? 0.f : 1.f / total);
#pragma unroll 1
                    for (int ch = ch0; ch < ch0 + chs; ch += 16) {
                        float x[16], o[2][16];
                        // (both streams' outputs are loaded, one that is not there too: its lanes' columns hold some number)
                        tc::tmem_load(o[0], tmem + F::kO + lanes + ch);
                        tc::tmem_load(o[1], tmem + F::kO + D + lanes + ch);
                        tc::tmem_wait_load(o);
#pragma unroll
                        for (int i = 0; i < 16; ++i) {
                            const float a = use_0 ? o[0][i] * mul_0 : 0.f, b = use_1 ? o[1][i] * mul_1 : 0.f;
                            x[i] = nothing ? 0.f : a + b;
                        }
                        if (mine) {
                            if (parts == 1) {
                                store(ch, x, f);
                            } else {
#pragma unroll
                                for (int i = 0; i < 16; ++i) __stcg(&W.o[slot][ch + i][r], x[i]);
                            }
                        }
                    }
                }
                if (*static_cast<volatile int *>(&S.nan_met[st.item]) != 0 && mine) {
                    // rare: NaN among values that only some rows attend to, read again from the cache
                    const int from = max(st.start, st.part_key0), to = min(st.stop, st.key0 + kTile);
#pragma unroll 1
                    for (int j = from; j < to; ++j) {
                        if (j >= st.common_from && j <= st.common_to) continue;
                        uint32_t sees[4];
                        row_keys(P, row, st.pos0, j, sees);
                        if (!(sees[0] & 1)) continue;
                        const int page = P.table[static_cast<int64_t>(st.seq) * P.max_blocks + (j >> P.page_shift)];
                        if (page < 0 || page >= P.num_pages) continue;
                        const int64_t at = ((static_cast<int64_t>(page) * P.Hkv + st.head) << P.page_shift) +
                                           (j & ((1 << P.page_shift) - 1));
#pragma unroll 1
                        for (int c = ch0; c < ch0 + chs; ++c) {
                            if ((P.v[at * D + c] & 0x7F) != 0x7F) continue;
                            if (parts == 1)
                                out[c] = narrow<E>(__int_as_float(0x7FC00000));
                            else
                                __stcg(&W.o[slot][c][r], __int_as_float(0x7FC00000));
                        }
                    }
                }
                tc::fence_before();
                if (took & 1) arrive(&S.o_free[0]), ++ended[0];
                if (took & 2) arrive(&S.o_free[1]), ++ended[1];
                if (parts > 1) {
                    // The part goes to the workspace; the CTA that brings the last one joins them, in the order of
                    // their keys whoever that is.
                    if ((pair || group == 0) && mine) __stcg(&W.ml[slot][r], make_float2(top, total));
                    __threadfence();
                    arrive(&S.meet);
                    if (!wait(&S.meet, meets++ & 1)) break;
                    if (tid == 0) {
                        S.last_part = atomicAdd(&W.arrived[first_cta], 1) == parts - 1;
                        __threadfence();
                    }
                    arrive(&S.meet);
                    if (!wait(&S.meet, meets++ & 1)) break;
                    if (*static_cast<volatile int *>(&S.last_part)) {
                        __threadfence();
                        if (tid == 0) W.arrived[first_cta] = 0;
                        if (mine) {
                            float high = kNothing, all = 0.f;
#pragma unroll 4
                            for (int i = 0; i < parts; ++i) {
                                const float2 v = __ldcg(&W.ml[slot_of(first_cta + i)][r]);
                                const float to = fmaxf(high, v.x);
                                all = fmaf(v.y, ex2(v.x - to), all * ex2(high - to));
                                high = to;
                            }
                            const float inv = all == 0.f ? 0.f : 1.f / all;
#pragma unroll 1
                            for (int ch = ch0; ch < ch0 + chs; ch += 32) {
                                float x[32];
#pragma unroll
                                for (int i = 0; i < 32; ++i) x[i] = 0.f;
#pragma unroll 1
                                for (int i = 0; i < parts; i += 2) {  // two parts' loads under way together
                                    const int one = slot_of(first_cta + i), two = slot_of(first_cta + min(i + 1, parts - 1));
                                    float a[32], b[32];
#pragma unroll
                                    for (int e = 0; e < 32; ++e) a[e] = __ldcg(&W.o[one][ch + e][r]), b[e] = __ldcg(&W.o[two][ch + e][r]);
                                    const float f = ex2(__ldcg(&W.ml[one][r]).x - high) * inv;
                                    const float g = i + 1 < parts ? ex2(__ldcg(&W.ml[two][r]).x - high) * inv : 0.f;
#pragma unroll
                                    for (int e = 0; e < 32; ++e) x[e] = fmaf(a[e], f, i + 1 < parts ? fmaf(b[e], g, x[e]) : x[e]);
                                }
                                store(ch, x, 1.f), store(ch + 16, x + 16, 1.f);
                            }
                        }
                    }
                }
                // NaN that was met concerns this item alone: cleared once both groups have looked, before the number is used again
                if (*static_cast<volatile int *>(&S.nan_met[st.item]) != 0) {
                    arrive(&S.meet);
                    if (!wait(&S.meet, meets++ & 1)) break;
                    if (tid == 0) S.nan_met[st.item] = 0;
                    arrive(&S.meet);
                    if (!wait(&S.meet, meets++ & 1)) break;
                }
            }
            arrive(&S.step_free[it % kSteps]);
            if (++k_slot == F::kKeys) k_slot = 0;
        }
    } else if (warp < 12) {
        // ---- the queries' digits, and V's halves -------------------------------------------
        const int w4 = warp - 8, t4 = tid - 256;
        // A query row has D / 8 lanes, 8 channels each, and a warp a batch of rows at a time; the next batch is under way
        // meanwhile.
        constexpr int kLanes = D / 8, kAtOnce = 32 / kLanes, kBatch = 4;
        // scores of scale 0 are those of digits that are all 0
        const float sign = P.scale < 0.f ? -1.f : (P.scale > 0.f ? 1.f : 0.f), size = P.scale == 0.f ? 1.f : fabsf(P.scale);
        const int most = min(126, 126 + ilogbf(size));
        const int sub = lane / kLanes, chunk = lane % kLanes;
        int items = 0;
        for (int it = 0;; ++it) {
            const int flags = open_step(it);
            if (!(flags & kLive)) break;
            const Step &st = S.step[it % kSteps];
            if (flags & kBegins) {
                const int rows = st.rows, row0 = st.row0, token0 = st.token0, head0 = st.head * P.G;
                constexpr int kRows = kAtOnce * kBatch;  // of a batch
                uint4 x[kBatch];
                auto load = [&](int r0) {
#pragma unroll
                    for (int i = 0; i < kBatch; ++i) {
                        const int r = r0 + i * kAtOnce + sub, row = row0 + r, node = node_of(P, row);
                        const E *q = static_cast<const E *>(P.q) + (token0 + node) * P.q_stride +
                                     static_cast<int64_t>(head0 + row - node * P.G) * D + chunk * 8;
                        x[i] = r < rows ? __ldg(reinterpret_cast<const uint4 *>(q)) : make_uint4(0, 0, 0, 0);
                    }
                };
                load(w4 * kRows);
                if (items > 0 && !wait(&S.q_free, (items - 1) & 1)) break;
#pragma unroll 1
                for (int r0 = w4 * kRows; r0 < rows; r0 += 4 * kRows) {
                    uint4 now[kBatch];
#pragma unroll
                    for (int i = 0; i < kBatch; ++i) now[i] = x[i];
                    if (r0 + 4 * kRows < rows) load(r0 + 4 * kRows);
                    uint32_t top[kBatch];  // without their signs, halves of either kind order as whole numbers
#pragma unroll
                    for (int i = 0; i < kBatch; ++i) {
                        const uint32_t t = __vmaxu2(__vmaxu2(now[i].x & 0x7FFF7FFFu, now[i].y & 0x7FFF7FFFu),
                                                    __vmaxu2(now[i].z & 0x7FFF7FFFu, now[i].w & 0x7FFF7FFFu));
                        top[i] = max(t & 0xFFFFu, t >> 16);
                    }
#pragma unroll
                    for (int o = 1; o < kLanes; o <<= 1)
#pragma unroll
                        for (int i = 0; i < kBatch; ++i) top[i] = max(top[i], __shfl_xor_sync(kAll, top[i], o));
#pragma unroll
                    for (int i = 0; i < kBatch; ++i) {
                        const int r = r0 + i * kAtOnce + sub;
                        const uint16_t bits = static_cast<uint16_t>(top[i]);
                        const float largest = wide(*reinterpret_cast<const E *>(&bits));
                        const bool odd = !(largest <= kMost);
                        // The largest is brought into [128, 256): k = 7 - its exponent, but not so far that the factor of the
                        // scores, |scale| 2^-k, falls below the normal range.
                        const int e = static_cast<int>(__float_as_uint(largest) >> 23);
                        const int k = largest == 0.f ? 0 : min(134 - e, most);
                        const float up = sign * power(127 + k);
                        uint8_t *q_at = q_sh + (r >> 7) * (kDigits * F::kSlot) + tc::swizzled<D>(r & 127, chunk >> 1) + 8 * (chunk & 1);
                        const uint32_t *two = &now[i].x;
                        uint32_t digit[kDigits][2];
#pragma unroll
                        for (int c = 0; c < 4; ++c) {
                            // scaled, a channel is exact as a half down to 2^-14, far below where the digits end; what a digit
                            // leaves of it is exact
                            const E *v = reinterpret_cast<const E *>(&two[c]);
                            __half2 left = __floats2half2_rn(wide(v[0]) * up, wide(v[1]) * up);
#pragma unroll
                            for (int g = 0; g < kDigits; ++g) {
                                const uint32_t d = e4m3x2_of_halves(left), back = halves_of_e4m3x2(d);
                                left = __hsub2(left, *reinterpret_cast<const __half2 *>(&back));
                                digit[g][c / 2] = c % 2 == 0 ? d : digit[g][c / 2] | (d << 16);
                            }
                        }
                        if (r < rows) {
#pragma unroll
                            for (int g = 0; g < kDigits; ++g)
                                *reinterpret_cast<uint2 *>(q_at + g * F::kSlot) = make_uint2(digit[g][0], digit[g][1]);
                            if (chunk == 0) S.q_factor[st.item][r] = odd ? __int_as_float(0x7FC00000) : size * power(127 - k);
                        }
                    }
                }
                tc::fence_async_shared();
                arrive(&S.q_full);
                ++items;
            }
            const int slot = it % F::kValues, buf = it & 1;
            if (!wait(&S.v_full[slot], (it / F::kValues) & 1)) break;
            if (it >= 2 && !wait(&S.h_free[buf], ((it >> 1) - 1) & 1)) break;
            const uint8_t *from = v_sh + slot * F::kSlot;
            uint8_t *to = h_sh + buf * F::kHalves;
            const bool plain = flags & kWhole;
            constexpr int kChunks = D / 16;  // of a key
            // (a thread's keys are a multiple of 8 apart, so that the swizzle is the same for all)
            const int c = t4 % kChunks, own = t4 / kChunks;
            from += tc::swizzled<D>(own, c);
            // 64 channels to a block of 128-byte rows; lanes of one key store even and odd chunks, which are in other banks
            const int odd = c >> 2, j0 = (c & 3) * 2;
            uint8_t *to_1 = to + odd * (kTile * 128) + tc::swizzled<128>(own, j0 + odd);
            uint8_t *to_2 = to + odd * (kTile * 128) + tc::swizzled<128>(own, j0 + 1 - odd);
            bool met = false;
            uint4 next = *reinterpret_cast<const uint4 *>(from);
#pragma unroll 1
            for (int i = 0; i < kChunks; ++i) {
                const int key = i * (kTile / kChunks) + own;
                uint4 x = next;
                if (i + 1 < kChunks) next = *reinterpret_cast<const uint4 *>(from + (i + 1) * (kTile / kChunks * D));
                uint32_t *w = &x.x;
                if (!plain) {
                    // A weight of 0 times NaN is NaN: values that no row, or not every row, attends to are cleared of it.
                    // NaN that some rows do attend to is put back with the output.
                    const int j = st.key0 + key;
                    const bool seen = ((st.there >> (key >> 4)) & 1) && j >= st.start && j < st.stop;
                    if (!seen) {
                        x = make_uint4(0, 0, 0, 0);
                    } else if (j < st.common_from || j > st.common_to) {
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            // a byte is NaN iff its low seven bits are all set
                            const uint32_t nan = ((w[e] & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u;
                            if (nan) met = true, w[e] &= ~((nan >> 7) * 0xFFu);
                        }
                    }
                }
                uint32_t h[8];
#pragma unroll
                for (int e = 0; e < 4; ++e) h[2 * e] = halves_of_e4m3x2(w[e] & 0xFFFFu), h[2 * e + 1] = halves_of_e4m3x2(w[e] >> 16);
                const uint4 lo = make_uint4(h[0], h[1], h[2], h[3]), hi = make_uint4(h[4], h[5], h[6], h[7]);
                *reinterpret_cast<uint4 *>(to_1 + i * (kTile / kChunks * 128)) = odd ? hi : lo;
                *reinterpret_cast<uint4 *>(to_2 + i * (kTile / kChunks * 128)) = odd ? lo : hi;
            }
            if (met) atomicExch(&S.nan_met[st.item], 1);
            tc::fence_async_shared();
            __syncwarp();
            if (!(withheld(SSD_CHECK_VALUES, it) && w4 == 0)) tc::warp_arrive(&S.h_full[buf]);
            tc::warp_arrive(&S.v_empty[slot]);
            tc::warp_arrive(&S.step_free[it % kSteps]);
        }
    } else if (warp == 12) {
        // ---- TMA ------------------------------------------------------------------------
        int n = 0;
        for (;; ++n) {
            if (!(open_step(n) & kLive)) break;
            const Step &st = S.step[n % kSteps];
            const int groups = 1 << max(P.page_shift - 4, 0);  // of a page
            const bool mine = lane < kGroups && lane % groups == 0 && ((st.there >> lane) & 1);
            const int bytes = __popc(__ballot_sync(kAll, mine)) * (D << P.page_shift);
            const int y = mine ? (st.page[lane] * P.Hkv + st.head) << P.page_shift : 0;
            const int k_slot = n % F::kKeys, v_slot = n % F::kValues;
            if (n >= F::kKeys && !wait(&S.k_empty[k_slot], (n / F::kKeys - 1) & 1)) break;
            const bool copied = !withheld(SSD_CHECK_COPIES, n);
            if (copied) tc::warp_arrive_expect(&S.k_full[k_slot], static_cast<uint32_t>(bytes));
            __syncwarp();
            if (copied && mine) tc::tma_load_2d(k_sh + k_slot * F::kSlot + lane * (16 * D), &k_map, 0, y, &S.k_full[k_slot]);
            S.k_issued = n + 1;
            if (n >= F::kValues && !wait(&S.v_empty[v_slot], (n / F::kValues - 1) & 1)) break;
            tc::warp_arrive_expect(&S.v_full[v_slot], static_cast<uint32_t>(bytes));
            __syncwarp();
            if (mine) tc::tma_load_2d(v_sh + v_slot * F::kSlot + lane * (16 * D), &v_map, 0, y, &S.v_full[v_slot]);
            S.v_issued = n + 1;
            arrive(&S.step_free[n % kSteps]);
        }
    } else if (warp == 13) {
        // ---- MMA ------------------------------------------------------------------------
        const uint64_t k_desc = tc::matrix_desc(k_sh, D), q_desc = tc::matrix_desc(q_sh, D);
        const uint64_t h_desc = tc::matrix_desc_wide(h_sh, kTile * 128);
        constexpr uint32_t kScores = tc::mma_shape(kTile, false, false), kOutput = tc::mma_shape(D, false, true);
        constexpr int kLastOfStep = 1 << 16;
        // Of the passes whose scores have been issued and whose output has not, `behind` in number: their flags and steps, the
        // older one first.
        int behind = 0, flags_0 = 0, flags_1 = 0, step_0 = 0, step_1 = 0;
        int e = 0, ended_0 = 0, ended_1 = 0;  // passes whose scores have been issued; items that the streams have finished
        int halves = -1;  // last step whose values have been seen as halves
        auto output_ready = [&] {
            const int g = (e - behind) & 1, done = g ? ended_1 : ended_0;
            if (step_0 != halves) wait(&S.h_full[step_0 & 1], (step_0 >> 1) & 1);
            halves = step_0;
            if ((flags_0 & kFirst) && done > 0) wait(&S.o_free[g], (done - 1) & 1);
            return wait(&S.p_full[g], ((e - behind) >> 1) & 1);
        };
        auto output_issue = [&] {  // O += P V
            const int g = (e - behind) & 1, buf = step_0 & 1;
            const uint32_t o = tmem + F::kO + g * D, p = tmem + g * kTile;
            const uint64_t h = h_desc + (buf * F::kHalves >> 4);
            tc::warp_mma_f16_tmem(o, p, h, kOutput, !(flags_0 & kFirst));
#pragma unroll
            for (int k = 1; k < kTile / 16; ++k) tc::warp_mma_f16_tmem(o, p + 8 * k, h + (k * 16 * 128 >> 4), kOutput, true);
            if (flags_0 & kLastOfStep) tc::warp_mma_commit(&S.h_free[buf]);
            if (flags_0 & kLast) tc::warp_mma_commit(&S.o_full[g]);
        };
        auto output_done = [&] {
            if (flags_0 & kLast) {
                if ((e - behind) & 1)
                    ++ended_1;
                else
                    ++ended_0;
            }
            flags_0 = flags_1, step_0 = step_1;
            --behind;
        };
        auto flush = [&] {
#pragma unroll 1
            while (behind > 0) {
                if (!output_ready()) return false;
                tc::fence_after();
                output_issue();
                output_done();
            }
            return true;
        };
        int items = 0, k_slot = 0, k_phase = 0, t = 0, flags = open_step(0);
        for (int n = 0; flags & kLive;) {
            if (t == 0) {
                arrive(&S.step_free[n % kSteps]);
                // an item's first scores wait for its queries, and all of the item before can end meanwhile
                if ((flags & kBegins) && !(flush() && wait(&S.q_full, items++ & 1))) break;
            }
            // Pass e of stream e & 1: its scores lie where the weights of the stream's pass before are, whose output goes first.
            const bool last = t == 1 || !(flags & kPair), before = behind == 2;
            const int flags_next = last ? open_step(n + 1) : flags;
            if (before && !output_ready()) break;
            if (t == 0 && !wait(&S.k_full[k_slot], k_phase)) break;
            tc::fence_after();
            if (before) output_issue();
            const uint64_t q = q_desc + (t * kDigits * F::kSlot >> 4), k8 = k_desc + (k_slot * F::kSlot >> 4);
            const uint32_t s_at = tmem + (e & 1) * kTile;
#pragma unroll
            for (int d = 0; d < kDigits; ++d)
#pragma unroll
                for (int k = 0; k < D / 32; ++k)  // 32 channels further inside the swizzled rows
                    tc::warp_mma_e4m3(s_at, q + ((d * F::kSlot + k * 32) >> 4), k8 + (k * 32 >> 4), kScores, d + k > 0);
            if (!withheld(SSD_CHECK_SCORES, n)) tc::warp_mma_commit(&S.s_full[e & 1]);
            if (last && (flags & kEnds)) tc::warp_mma_commit(&S.q_free);
            if (before) output_done();
            if (behind == 0)
                flags_0 = flags | (last ? kLastOfStep : 0), step_0 = n;
            else
                flags_1 = flags | (last ? kLastOfStep : 0), step_1 = n;
            ++behind;
            ++e;
            n += last;
            t = last ? 0 : 1;
            if (last && ++k_slot == F::kKeys) k_slot = 0, k_phase ^= 1;
            flags = flags_next;
        }
        flush();
    } else if (warp == 14) {
        // ---- scout: items, pages and scales ahead of the others ---------------------------
        const int my_step = lane / kGroups, my_group = lane % kGroups;
        constexpr int kAtOnce = 32 / kGroups;  // steps whose pages the lanes look up together
        Part part;
        int s = 0, items = 0, event = 0;
        while (walk.next(P, part)) {
            if (__any_sync(kAll, gave_up())) break;
            const int high = part.pos0 + (part.row0 + part.rows - 1) / P.G;
            const int common_to = part.pos0 - 1, common_from = P.window > 0 && high >= P.window ? high + 1 - P.window : 0;
            const int32_t *table = P.table + static_cast<int64_t>(part.b) * P.max_blocks;
            const int key0 = part.step * kTile, passes = part.rows > kTile ? 2 : 1;
            // page of this lane's 16 keys in the steps from t on; -1 for what is no page, less for what is no place
            constexpr int kNoPlace = -2;
            auto look_up = [&](int t) {
                const int j = key0 + (t + my_step) * kTile + my_group * 16;
                // a page is there as a whole where any of its keys is wanted
                const int page0 = j >> P.page_shift << P.page_shift;
                const bool in = t + my_step < part.steps && page0 < part.stop && page0 + (1 << P.page_shift) > part.start;
                return in ? max(__ldg(table + (j >> P.page_shift)), -1) : kNoPlace;
            };
            int next = look_up(0);
            // The item's queries on their way: eight steps from now they are asked for, row by row, and from HBM each of
            // those waits would take 2000 clocks.
            for (int row = part.row0 + lane; row < part.row0 + part.rows; row += 32) {
                const int node = node_of(P, row);
                const E *q = static_cast<const E *>(P.q) + (part.first + node) * P.q_stride +
                             static_cast<int64_t>(part.head * P.G + row - node * P.G) * D;
                prefetch(q);
                if (D * sizeof(E) > 128) prefetch(q + 64);
                if (part.head * P.G + row - node * P.G == part.head * P.G) prefetch(P.mask + static_cast<int64_t>(part.first + node) * P.words);
            }
            for (int t0 = 0; t0 < part.steps; t0 += kAtOnce) {
                const int page = next;
                const bool there = page >= 0 && page < P.num_pages;
                float ks = 0.f, vs = 0.f;
                if (there) {
                    const int64_t block = static_cast<int64_t>(page) * P.Hkv + part.head;
                    ks = __ldg(P.ks + block);
                    vs = __ldg(P.vs + block);
                }
                if (page != kNoPlace && !there) report(P.dev_status, SSD_DEV_BAD_PAGE);
                if (t0 + kAtOnce < part.steps) next = look_up(t0 + kAtOnce);
                const bool finite = fabsf(vs) <= kMost;
                const float lv = finite ? lg2_of_any(fabsf(vs)) : __int_as_float(0x7FC00000);
                float k_most = ks;
#pragma unroll
                for (int o = 1; o < kGroups; o <<= 1) k_most = fmaxf(k_most, __shfl_xor_sync(kAll, k_most, o));
                const uint32_t there_all = __ballot_sync(kAll, there);
                // between 2^-100 and 2^100, and between 2^-kMostUnit and 2^kMostUnit
                const uint32_t fast_all = __ballot_sync(kAll, !there || (ks >= 7.9e-31f && ks <= 1.2e30f && fabsf(lv) <= kMostUnit && vs > 0.f));
                const int n = min(kAtOnce, part.steps - t0);
                for (int i = 0; i < n; ++i, ++s) {
                    const int slot = s % kSteps;
                    if (s >= kSteps) wait(&S.step_free[slot], (s / kSteps - 1) & 1);
                    if (__any_sync(kAll, gave_up())) break;
                    Step &st = S.step[slot];
                    if (my_step == i) {
                        st.page[my_group] = page;
                        st.scale[my_group] = there ? make_float4(ks, finite ? vs : __int_as_float(0x7FC00000), lv, __frcp_rn(vs))
                                                      : make_float4(1.f, 1.f, 0.f, 1.f);
                        if (my_group == 0) {
                            const int k0 = key0 + (t0 + i) * kTile;
                            const uint32_t mask = (there_all >> (i * kGroups)) & 0xFFu;
                            const int index = t0 + i, left = part.steps - 1 - index;
                            const bool whole = mask == 0xFFu && k0 >= common_from && k0 + kTile - 1 <= common_to;
                            const bool fast = ((fast_all >> (i * kGroups)) & 0xFFu) == 0xFFu;
                            st.flags = kLive | (passes == 2 ? kPair : 0) | (index == 0 ? kBegins : 0) | (left == 0 ? kEnds : 0) |
                                       (index < 3 - passes ? kFirst : 0) | (left < 3 - passes ? kLast : 0) | (whole ? kWhole : 0) |
                                       (fast ? kOrdinary : 0) | (event & 1 ? kStream : 0) | (part.steps == 1 ? kSingle : 0);
                            st.key0 = k0;
                            st.start = part.start, st.stop = part.stop;
                            st.common_from = common_from, st.common_to = common_to;
                            st.there = static_cast<int32_t>(mask);
                            st.item = items % kItems;
                            st.first_cta = part.first_cta, st.parts = part.parts;
                            st.seq = part.b, st.head = part.head, st.row0 = part.row0, st.rows = part.rows;
                            st.token0 = part.first, st.pos0 = part.pos0;
                            st.part_key0 = key0;
                            st.k_most = k_most;
                        }
                    }
                    event += passes;
                    if (withheld(SSD_CHECK_STEPS, s))
                        __syncwarp();
                    else
                        arrive(&S.step_full[slot]);
                }
            }
            ++items;
        }
        // the end
        const int slot = s % kSteps;
        if (s >= kSteps) wait(&S.step_free[slot], (s / kSteps - 1) & 1);
        if (!__any_sync(kAll, gave_up())) {
            if (lane == 0) S.step[slot].flags = 0;
            arrive(&S.step_full[slot]);
        }
    }
    __syncwarp();
    tc::fence_before();
    __syncthreads();
    tc::fence_after();
    if (gave_up()) {
        if (tid == 0) report(P.dev_status, SSD_DEV_TIMEOUT);
        // Some role left early, perhaps after the ones that issue copies and products had left: what they issued still
        // has to end before the CTA does.
        if (warp == 12) {
            const int k = S.k_issued, v = S.v_issued;
#pragma unroll 1
            for (int x = max(0, k - F::kKeys); x < k; ++x) drain_phase<kWait>(&S.k_full[x % F::kKeys], (x / F::kKeys) & 1);
#pragma unroll 1
            for (int x = max(0, v - F::kValues); x < v; ++x) drain_phase<kWait>(&S.v_full[x % F::kValues], (x / F::kValues) & 1);
        }
        if (warp == 13) {
            // (of the thread that issued them: a commit is of its own thread's products)
            tc::warp_mma_commit(&S.drained);
            drain_phase<kWait>(&S.drained, 0);
        }
    }
    if (warp == 13) tc::tmem_free(tmem, 512);
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

template <class F, bool kOwn, bool kChecked = false>
int tree_run(const TreeParams &P, const CUtensorMap &k_map, const CUtensorMap &v_map, const Device &dev, int ctas, cudaStream_t stream) {
    auto *kernel = tree_kernel<F, kOwn, kChecked>;
    constexpr int dyn = F::kBytes + static_cast<int>(sizeof(Shared<F>)) + (kOwn ? 4 * kInside + 2 : kInside + 1) * 4;
    static_assert(dyn <= 227 * 1024);
    if (dyn > dev.smem_cta) return SSD_ERR_UNSUPPORTED;
    static std::atomic<uint64_t> ready{0};  // devices on which this kernel may take that much
    const uint64_t bit = 1ull << (dev.id & 63);
    if (!(ready.load(std::memory_order_relaxed) & bit)) {
        cudaFuncAttributes attr;
        if (cudaFuncGetAttributes(&attr, kernel) != cudaSuccess ||
            cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, dyn) != cudaSuccess) {
            cudaGetLastError();
            return SSD_ERR_CUDA;
        }
        // the registers that the softmax warps take over have to be there
        if (attr.numRegs < kRegisters) return SSD_ERR_UNSUPPORTED;
        ready.fetch_or(bit, std::memory_order_relaxed);
    }
    kernel<<<static_cast<unsigned>(ctas), kTreeThreads, static_cast<size_t>(dyn), stream>>>(P, k_map, v_map);
    return launched();
}

template <class F>
int tree_launch(TreeParams P, const CUtensorMap &k_map, const CUtensorMap &v_map, const Device &dev, cudaStream_t stream) {
    int ctas = dev.sms;
    if (ctas > kMaxCtas) ctas = kMaxCtas;
    P.inside = P.B <= kInside && static_cast<int64_t>(P.max_new) * P.G <= kMaxRows;
    const int64_t most = static_cast<int64_t>(P.T) * P.G / kMaxRows + P.B;
    P.most_pairs = static_cast<int>(most < kMaxPairs ? most : kMaxPairs);
    if (P.withheld) {
        if constexpr (__is_same(typename F::E, __nv_bfloat16) && F::D == 64)
            if (P.inside) return tree_run<F, false, true>(P, k_map, v_map, dev, ctas, stream);
        return SSD_ERR_UNSUPPORTED;
    }
    if (P.inside) return tree_run<F, false>(P, k_map, v_map, dev, ctas, stream);
    // A schedule in the workspace takes a launch of its own (6 sequences of up to 509 nodes: 58.5 us, and 62.6 with it).
    if (most <= kInside) return tree_run<F, true>(P, k_map, v_map, dev, ctas, stream);
    if (most > kMaxPairs) return SSD_ERR_UNSUPPORTED;
    schedule_kernel<<<1, kScheduleThreads, 0, stream>>>(P, ctas);
    if (launched() != SSD_OK) return SSD_ERR_CUDA;
    return tree_run<F, false>(P, k_map, v_map, dev, ctas, stream);
}

int attend_tree(const void *q, int dtype, int64_t q_stride, const void *k_cache, const void *v_cache, const float *k_scale,
                const float *v_scale, int num_pages, int page_size, int Hq, int Hkv, int D, const int32_t *block_table,
                int max_blocks, const int32_t *cu_new, const int32_t *kv_len, const int32_t *mask, int B, int T, int max_new,
                float sm_scale, int window, void *out, void *workspace, size_t workspace_bytes, int32_t *dev_status,
                void *stream, int withheld) {
    if (dtype != SSD_BF16 && dtype != SSD_F16) return SSD_ERR_DTYPE;
    if (B < 1 || T < 0 || max_new < 1 || num_pages < 1 || max_blocks < 1 || Hkv < 1 || Hq < 1 || Hq % Hkv != 0 ||
        window < 0 || !kv_page_size_ok(page_size) || (D != 64 && D != 128))
        return SSD_ERR_INVALID_ARG;
    const float scale = sm_scale * kLog2e;
    if (!(scale - scale == 0.f)) return SSD_ERR_INVALID_ARG;
    if (!k_cache || !v_cache || !k_scale || !v_scale || !block_table || !cu_new || !kv_len || (T > 0 && (!q || !out || !mask)))
        return SSD_ERR_INVALID_ARG;
    if (!aligned(k_cache, 16) || !aligned(v_cache, 16)) return SSD_ERR_INVALID_ARG;
    if (T > 0 && (!aligned(q, 16) || !aligned(out, 16))) return SSD_ERR_INVALID_ARG;
    if (T > 1 && (q_stride < static_cast<int64_t>(Hq) * D || q_stride % 8 != 0)) return SSD_ERR_INVALID_ARG;
    if (!workspace || !aligned(workspace, 256) || workspace_bytes < ssd_kv_tree_workspace_size()) return SSD_ERR_WORKSPACE;
    if (static_cast<int64_t>(num_pages) * page_size > 0x7FFFFFFF ||
        static_cast<int64_t>(num_pages) * Hkv > 0x7FFFFFFF / page_size ||
        static_cast<int64_t>(B) * max_blocks > 0x7FFFFFFF || static_cast<int64_t>(max_blocks) * page_size > 0x7FFFFFFF / 2 ||
        B > SSD_KV_MAX_B || max_new > SSD_TREE_MAX)
        return SSD_ERR_UNSUPPORTED;
    // Units of all items, which the schedule counts in 32 bits: steps of 128 keys, the last one begun, and an item's start.
    const int64_t row_blocks = static_cast<int64_t>(T < 1 ? 1 : T) * (Hq / Hkv) / kMaxRows + B;
    if (row_blocks * Hkv > 0x7FFFFFFF / (static_cast<int64_t>(max_blocks) * page_size / kTile + 1 + kItemCost)) return SSD_ERR_UNSUPPORTED;
    if (T == 0) return SSD_OK;
    TreeParams P{};
    P.q = q, P.q_stride = q_stride;
    P.v = static_cast<const uint8_t *>(v_cache);
    P.ks = k_scale, P.vs = v_scale;
    P.num_pages = num_pages, P.page_shift = log2_of(page_size);
    P.Hq = Hq, P.Hkv = Hkv, P.G = Hq / Hkv;
    P.g_shift = (P.G & (P.G - 1)) == 0 ? log2_of(P.G) : -1;
    P.table = block_table, P.max_blocks = max_blocks;
    P.cu = cu_new, P.kv_len = kv_len, P.mask = mask, P.words = (max_new + 31) / 32;
    P.B = B, P.T = T, P.max_new = max_new < T ? max_new : T;
    P.scale = scale, P.window = window, P.out = out;
    P.ws = static_cast<Workspace *>(workspace);
    P.dev_status = dev_status;
    P.withheld = withheld;
    Device dev;
    if (device_limits(&dev) != SSD_OK) return SSD_ERR_CUDA;
    CUtensorMap k_map, v_map;
    const uint64_t rows = static_cast<uint64_t>(num_pages) * Hkv * page_size;
    if (!tc::encode_rows(&k_map, k_cache, rows, D, page_size) || !tc::encode_rows(&v_map, v_cache, rows, D, page_size))
        return SSD_ERR_CUDA;
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (dtype == SSD_BF16)
        return D == 64 ? tree_launch<Form<__nv_bfloat16, 64>>(P, k_map, v_map, dev, s)
                       : tree_launch<Form<__nv_bfloat16, 128>>(P, k_map, v_map, dev, s);
    return D == 64 ? tree_launch<Form<__half, 64>>(P, k_map, v_map, dev, s) : tree_launch<Form<__half, 128>>(P, k_map, v_map, dev, s);
}

}  // namespace
}  // namespace ssd

extern "C" size_t ssd_kv_tree_workspace_size(void) { return (sizeof(ssd::Workspace) + 255) / 256 * 256; }

extern "C" int ssd_kv_attend_tree(const void *q, int dtype, int64_t q_stride, const void *k_cache, const void *v_cache,
                                  const float *k_scale, const float *v_scale, int num_pages, int page_size, int Hq,
                                  int Hkv, int D, const int32_t *block_table, int max_blocks, const int32_t *cu_new,
                                  const int32_t *kv_len, const int32_t *mask, int B, int T, int max_new, float sm_scale,
                                  int window, void *out, void *workspace, size_t workspace_bytes, int32_t *dev_status,
                                  void *stream) {
    return ssd::attend_tree(q, dtype, q_stride, k_cache, v_cache, k_scale, v_scale, num_pages, page_size, Hq, Hkv,
                            D, block_table, max_blocks, cu_new, kv_len, mask, B, T, max_new, sm_scale, window,
                            out, workspace, workspace_bytes, dev_status, stream, 0);
}

extern "C" int ssd_check_tree_timeout(int withheld, const void *q, int dtype, int64_t q_stride, const void *k_cache,
                                      const void *v_cache, const float *k_scale, const float *v_scale, int num_pages,
                                      int page_size, int Hq, int Hkv, int D, const int32_t *block_table, int max_blocks,
                                      const int32_t *cu_new, const int32_t *kv_len, const int32_t *mask, int B, int T,
                                      int max_new, float sm_scale, int window, void *out, void *workspace,
                                      size_t workspace_bytes, int32_t *dev_status, void *stream) {
    if (withheld < SSD_CHECK_STEPS || withheld > SSD_CHECK_SCORES) return SSD_ERR_INVALID_ARG;
    return ssd::attend_tree(q, dtype, q_stride, k_cache, v_cache, k_scale, v_scale, num_pages, page_size, Hq, Hkv,
                            D, block_table, max_blocks, cu_new, kv_len, mask, B, T, max_new, sm_scale, window,
                            out, workspace, workspace_bytes, dev_status, stream, withheld);
}
