// ssd_sample.cu -- one token per logit row under temperature, top-k, top-p and min-p
// (sm_103a).
//
// What is kept is a prefix of the ranking (logit desc, id asc), so it is described by its
// last value and, among tokens of that value, its last id.
//
// A cluster of CTAs takes a row: each holds one slice in shared memory, read from HBM once,
// and every pass after that runs on chip.  A limit (k tokens, or a share of the weight) is
// found on the distance d = max - z, whose float bits order the tokens: a histogram over 512
// ranges of those bits, of counts or of exact weights, names the range that the limit falls
// into, and the next one divides that range, until it holds at most 256 tokens, which are
// ranked against one another, or tokens of one value, which rank by id.  Every CTA adds up
// the cluster's histograms itself, so that one cluster barrier does for each.
//
// Weights.  w = exp((z - m) / tau) = 2^t, t = d * c with d = z - m and c = log2(e) / tau
// both carried as two floats, so that t is exact to about 2^-45 of itself.  t is split
// into k / 32 + g, g to 2^-31: a 32-entry table of 2^(i/32) (one entry per lane, read by shuffle) times
// a polynomial of 2^g - 1, |g| <= 1/64, gives 28 significant bits, which are shifted into
// 64-bit fixed point with 43 bits after the point.  Sums of those are exact: they depend
// on no order, a prefix and a total agree to the last bit, and the rank or id at which a
// sum passes its limit is decided as the real numbers would, but for cases closer than
// 2^-28 of a weight.
//
// What bounds it: some 35 instructions for each weight, and 1 to 2 us for each cluster
// barrier, of which a limit takes two to four.  256 rows of 128256 bf16 logits, captured into
// a graph with L2 flushed: 89 us without limits, 106 top-k, 194 top-p, 64 min-p (the tokens
// below the limit need no weight), 106 mixed; the bytes would take 10.  Two CTAs to an SM: one
// computes while the other waits.  Clusters of 8, three CTAs to an SM and CTAs of 1024
// threads were all slower.
#include <cooperative_groups.h>
#include <cuda_bf16.h>

#include <atomic>
#include <cfloat>

#include "ssd_kv.h"
#include "ssd_device.cuh"

namespace ssd {
namespace {

namespace cg = cooperative_groups;

constexpr int kSampleThreads = 512;
constexpr int kSampleWarps = kSampleThreads / 32;
constexpr int kBins = kSampleThreads;  // a thread adds up one bin
constexpr int kList = 256;
constexpr uint32_t kAll = 0xFFFFFFFFu;
// The first histogram: 32 ranges for each power of two of d from 2^-6 on, what is nearer and
// what is farther in one range each.
constexpr uint32_t kNear = 0x3C800000u, kFirstShift = 18, kInfinite = 0x7F800000u;

struct SampleParams {
    const void *logits;
    int rows, V;
    int64_t ld;
    const float *tau;
    const int32_t *top_k;
    const float *top_p, *min_p, *u;
    int32_t *tokens;
    float *prob;
    void *filtered;
    int32_t *dev_status;
    int slice;    // 16-byte vectors of a CTA
    int aligned;  // rows start on 16-byte boundaries
};

// 2^t in fixed point, t = (z - m) * (c_hi + c_lo) <= 0.  All lanes call; `table` is this
// lane's 2^(lane/32) in units of 2^-27.
struct Weigher {
    float m, c_hi, c_lo;
    uint32_t table;
    // The weight as `value` * 2^-(27 + shift), 2^27 <= value < 2^28; below 2^-60, and at -inf, shift passes 59 and
    // `value` may be anything.
    __device__ __forceinline__ void parts(float z, uint32_t &value, int &shift) const {
        const float d = z - m;
        // what the subtraction rounded off, exact (m >= z; both finite)
        const float bb = d - z;
        const float err = (z - (d - bb)) + (-m - bb);
        // t rounded to 1/32: `near` is so large that its last bit stands for that
        const float near = 393216.f;  // 1.5 * 2^18
        const float kn = fmaxf(fmaf(d, c_hi, near), near - 64.f);
        const int k = __float_as_int(kn) - __float_as_int(near);
        // what that leaves of t, from the product itself
        const float g = fmaf(err, c_hi, fmaf(d, c_lo, fmaf(d, c_hi, near - kn)));
        // (2^g - 1) = g (ln2 + g (ln2^2/2 + g (ln2^3/6 + g ln2^4/24)))
        float q = fmaf(g, 0.0096181291f, 0.0555041087f);
        q = fmaf(g, q, 0.2402265070f);
        q = fmaf(g, q, 0.6931471806f) * g;
        const uint32_t base = __shfl_sync(0xFFFFFFFFu, table, k & 31);
        // base as a float, cut off at 24 bits: its part of the product ends 2^-29 below
        const float rough = __uint_as_float((base >> 4) + 0x4C800000u);
        const float magic = 12582912.f;  // 1.5 * 2^23: the sum's low bits are the rounded value
        const int more = __float_as_int(fmaf(rough, q, magic)) - __float_as_int(magic);
        value = base + static_cast<uint32_t>(more);
        shift = -(k >> 5);
    }
    // (value << 16) >> shift; shl and shr give 0 for counts from 32 on, so that no case is told apart.
    __device__ __forceinline__ uint64_t operator()(float z) const {
        uint32_t value, high, low, small;
        int shift;
        parts(z, value, shift);
        asm("shr.b32 %0, %1, %2;" : "=r"(high) : "r"(value), "r"(16 + shift));
        asm("shl.b32 %0, %1, %2;" : "=r"(low) : "r"(value), "r"(16 - shift));
        asm("shr.b32 %0, %1, %2;" : "=r"(small) : "r"(value), "r"(shift - 16));
        return static_cast<uint64_t>(high) << 32 | (low | small);
    }
};

// 2^(i / 32) in units of 2^-27.
__device__ const uint32_t kPowers[32] = {
    134217728u, 137156714u, 140160054u, 143229160u,
    146365470u, 149570457u, 152845623u, 156192507u,
    159612677u, 163107740u, 166679334u, 170329136u,
    174058859u, 177870251u, 181765103u, 185745240u,
    189812531u, 193968884u, 198216250u, 202556621u,
    206992033u, 211524568u, 216156353u, 220889561u,
    225726413u, 230669177u, 235720175u, 240881774u,
    246156398u, 251546522u, 257054673u, 262683438u,};

// What is kept: values above `last`, or equal to it with an id up to `id`; and values >= `least`.
struct Kept {
    float last;
    int id;
    float least;
    __device__ __forceinline__ bool operator()(float z, int i) const {
        return (z > last || (z == last && i <= id)) && z >= least;
    }
    // no value above this is left out, none below it kept
    __device__ __forceinline__ float border() const { return fmaxf(last, least); }
};

// The same for the tokens of a vector at once (and not -inf): values from `upto` on for ids up to `id`, from `after` on
// for the rest.
struct Bounds {
    float upto, after;
    int id;
    __device__ __forceinline__ explicit Bounds(const Kept &k)
        : upto(fmaxf(k.border(), -FLT_MAX)), after(fmaxf(fmaxf(nextafterf(k.last, INFINITY), k.least), -FLT_MAX)), id(k.id) {}
    template <int kVec>
    __device__ __forceinline__ uint32_t mask(const float (&z)[kVec], int first) const {
        uint32_t a = 0, b = 0;
#pragma unroll
        for (int e = 0; e < kVec; ++e) {
            a |= z[e] >= upto ? 1u << e : 0u;
            b |= z[e] >= after ? 1u << e : 0u;
        }
        const uint32_t low = (1u << min(max(id - first + 1, 0), kVec)) - 1u;
        return (a & low) | (b & ~low);
    }
};

// Largest of a vector's values (NaN left out).
template <class D>
__device__ __forceinline__ float vector_max(const uint4 &w);
template <>
__device__ __forceinline__ float vector_max<F32Tag>(const uint4 &w) {
    return fmaxf(fmaxf(__uint_as_float(w.x), __uint_as_float(w.y)), fmaxf(__uint_as_float(w.z), __uint_as_float(w.w)));
}
template <>
__device__ __forceinline__ float vector_max<BF16Tag>(const uint4 &w) {
    auto two = [](uint32_t x) { return *reinterpret_cast<const __nv_bfloat162 *>(&x); };
    const __nv_bfloat162 m = __hmax2(__hmax2(two(w.x), two(w.y)), __hmax2(two(w.z), two(w.w)));
    return __bfloat162float(__hmax(__low2bfloat16(m), __high2bfloat16(m)));
}
// Whether any of a vector's values is NaN: the maximum that passes NaN on.
template <class D>
__device__ __forceinline__ bool vector_nan(const uint4 &w);
template <>
__device__ __forceinline__ bool vector_nan<F32Tag>(const uint4 &w) {
    const float a = __uint_as_float(w.x), b = __uint_as_float(w.y), c = __uint_as_float(w.z), d = __uint_as_float(w.w);
    return a != a || b != b || c != c || d != d;
}
template <>
__device__ __forceinline__ bool vector_nan<BF16Tag>(const uint4 &w) {
    auto two = [](uint32_t x) { return *reinterpret_cast<const __nv_bfloat162 *>(&x); };
    const __nv_bfloat162 m = __hmax2_nan(__hmax2_nan(two(w.x), two(w.y)), __hmax2_nan(two(w.z), two(w.w)));
    return isnan(__bfloat162float(__low2bfloat16(m))) || isnan(__bfloat162float(__high2bfloat16(m)));
}

struct Histogram {
    uint32_t count[kBins];
    uint2 mass[kBins];  // weights: 64 bits in two words
};

struct Shared {
    Histogram hist[2];
    uint64_t list[kList];    // this CTA's tokens of the range
    uint64_t ranked[kList];  // the cluster's
    uint64_t ranked_weight[kList];
    uint64_t sums[2][2][kSampleWarps];  // two words of each warp, published to the cluster in turn
    uint64_t stretches[kSampleWarps];   // sums over the warps' stretches
    uint64_t best[kSampleWarps];
    uint64_t inbox[2][16];  // a word from each CTA of the cluster
    int listed;
    int result;
    uint64_t red[kSampleWarps];
    uint64_t found_above, goal, target;
    uint32_t found_bin, found_in;
    double drop;  // tau log(min_p)
};

template <class D>
__device__ __forceinline__ void store_logit(void *p, int64_t i, float v);
template <>
__device__ __forceinline__ void store_logit<F32Tag>(void *p, int64_t i, float v) {
    static_cast<float *>(p)[i] = v;
}
template <>
__device__ __forceinline__ void store_logit<BF16Tag>(void *p, int64_t i, float v) {
    static_cast<__nv_bfloat16 *>(p)[i] = __float2bfloat16(v);
}

template <class D>
struct Row {
    static constexpr int kVec = D::kVec;
    const SampleParams &P;
    Shared &S;
    const uint4 *slice;
    cg::cluster_group cluster;
    int ctas, rank, first_id;  // id of the slice's first token
    int vectors;               // of the slice
    float top = -INFINITY;     // of this thread's vectors
    int turn = 0;  // which of the two sets of words is next
    float m;
    Weigher weigh;

    __device__ __forceinline__ Row(const SampleParams &p, Shared &s, const uint4 *sl)
        : P(p), S(s), slice(sl), cluster(cg::this_cluster()) {
        ctas = static_cast<int>(cluster.num_blocks());
        rank = static_cast<int>(cluster.block_rank());
        first_id = rank * P.slice * kVec;
        const int left = P.V - first_id;
        vectors = left <= 0 ? 0 : min(P.slice, (left + kVec - 1) / kVec);
    }
    // A vector of the slice, of -inf where it is none of the scan's.
    __device__ __forceinline__ uint4 vector(int v, int to) const {
        constexpr uint32_t kNone = kVec == 4 ? 0xFF800000u : 0xFF80FF80u;
        return v < to ? slice[v] : make_uint4(kNone, kNone, kNone, kNone);
    }
    // fn(vector, index, there) for vectors [from, to) of the slice in steps of `step`, whole warps at a time; those
    // whose largest logit is below `border` are passed over where a warp has no other.
    template <class Fn>
    __device__ __forceinline__ void scan(int from, int to, int step, int offset, float border, Fn &&fn) {
        for (int v0 = from; v0 < to; v0 += step) {
            const int v = v0 + offset;
            const uint4 w = vector(v, to);
            if (__any_sync(kAll, v < to && vector_max<D>(w) >= border)) fn(w, v, v < to);
        }
    }
    // Element e of a vector, e not known when compiling.
    __device__ __forceinline__ static float pick(const uint4 &w, int e) {
        if (kVec == 4) return __uint_as_float(e & 2 ? (e & 1 ? w.w : w.z) : (e & 1 ? w.y : w.x));
        const uint32_t two = e & 4 ? (e & 2 ? w.w : w.z) : (e & 2 ? w.y : w.x);
        return __uint_as_float(e & 1 ? two & 0xFFFF0000u : two << 16);
    }
    // fn(z, id, there) for the tokens of the slice.
    template <class Fn>
    __device__ __forceinline__ void each(float border, Fn &&fn) {
        scan(0, vectors, kSampleThreads, static_cast<int>(threadIdx.x), border, [&](const uint4 &w, int v, bool in) {
            float z[kVec];
            decode_vec<D>(w, z);
#pragma unroll
            for (int e = 0; e < kVec; ++e) {
                const int id = first_id + v * kVec + e;
                fn(z[e], id, in && id < P.V);
            }
        });
    }
    // Whether a warp's tokens are all one value.
    __device__ __forceinline__ static bool alike(const uint4 &w) {
        const uint32_t x = __shfl_sync(kAll, w.x, 0);
        return __all_sync(kAll, w.x == x && w.y == x && w.z == x && w.w == x && (kVec == 4 || x >> 16 == (x & 0xFFFFu)));
    }
    // add(z, weight, times) for the tokens of a vector in mask(z, first id), which takes none of -inf.  Where few are,
    // each lane goes from one of its own to the next, and the warp weighs as often as its fullest lane has any; where
    // a warp's tokens are all one value, lane 0 adds them all at once.
    template <class Mask, class Add>
    __device__ __forceinline__ void weigh_vector(const uint4 &w, int v, Mask &&mask_of, Add &&add) {
        float z[kVec];
        decode_vec<D>(w, z);
        uint32_t mask = mask_of(z, first_id + v * kVec);
        const int most = static_cast<int>(__reduce_max_sync(kAll, static_cast<uint32_t>(__popc(mask))));
        if (most == 0) return;
        if (most * 4 <= kVec * 3) {
            for (int i = 0; i < most; ++i) {
                const bool here = mask != 0;
                const float x = here ? pick(w, __ffs(mask) - 1) : m;
                mask &= mask - 1;
                const uint64_t weight = weigh(x);
                if (here) add(x, weight, 1u);
            }
            return;
        }
        if (alike(w) && __all_sync(kAll, mask == (1u << kVec) - 1u)) {
            const uint64_t weight = weigh(z[0]);
            if ((threadIdx.x & 31) == 0) add(z[0], weight * (32u * kVec), 32u * kVec);
            return;
        }
#pragma unroll
        for (int e = 0; e < kVec; ++e) {
            const uint64_t weight = weigh(z[e]);
            if ((mask >> e) & 1) add(z[e], weight, 1u);
        }
    }
    // add(z, weight, times) for every token of vectors [from, to): no test of any, as what lies beyond them or beyond
    // the row is -inf, whose weight is 0.
    template <class Add>
    __device__ __forceinline__ void weigh_all(int from, int to, int step, int offset, Add &&add) {
        for (int v0 = from; v0 < to; v0 += step) {
            const uint4 w = vector(v0 + offset, to);
            float z[kVec];
            decode_vec<D>(w, z);
            if (alike(w)) {
                const uint64_t weight = weigh(z[0]);
                if ((threadIdx.x & 31) == 0) add(z[0], weight * (32u * kVec), 32u * kVec);
                continue;
            }
#pragma unroll
            for (int e = 0; e < kVec; ++e) add(z[e], weigh(z[e]), 1u);
        }
    }
    __device__ __forceinline__ uint32_t distance(float z) const { return __float_as_uint(m - z); }
    // A value that every token nearer than d exceeds: m - d less what the distances and this difference are rounded by.
    __device__ __forceinline__ float nearest(uint32_t d) const {
        const float x = __uint_as_float(min(d, 0x7F7FFFFFu));
        return m - x - (fabsf(m) + x) * 1e-6f;
    }

    // What each warp of the cluster published in word `which`, joined by op(cta, word) over the lanes of every warp:
    // no second stage in the CTA, and all the loads are under way together.
    template <class Op>
    __device__ __forceinline__ void gather(const uint64_t *words, Op &&op) {
        const int lane = static_cast<int>(threadIdx.x & 31);
#pragma unroll 4
        for (int i = lane; i < ctas * kSampleWarps; i += 32)
            op(i / kSampleWarps, cluster.map_shared_rank(words, i / kSampleWarps)[i % kSampleWarps]);
    }
    // Sends this CTA's word, join() in the threads that send it, to every CTA of the cluster, and returns CTA `lane`'s (0
    // in lanes beyond them).  What is read afterwards is at hand, and no CTA is read after the barrier, so that none
    // has to wait for another to leave.
    template <class Join>
    __device__ __forceinline__ uint64_t exchange(Join &&join) {
        const int t = static_cast<int>(threadIdx.x), lane = t & 31;
        __syncthreads();
        if (t < ctas) *cluster.map_shared_rank(&S.inbox[turn][rank], t) = join();
        cluster.sync();
        const uint64_t x = lane < ctas ? S.inbox[turn][lane] : 0;
        turn ^= 1;
        return x;
    }
    __device__ __forceinline__ uint64_t warp_total(uint64_t x) {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(kAll, x, o);
        return x;
    }
    // Sum over the cluster; every thread gets it.
    __device__ __forceinline__ uint64_t cluster_sum(uint64_t a) {
        a = warp_total(a);
        if ((threadIdx.x & 31) == 0) S.sums[turn][0][threadIdx.x >> 5] = a;
        cluster.sync();
        uint64_t total = 0;
        gather(&S.sums[turn][0][0], [&](int, uint64_t x) { total += x; });
        turn ^= 1;
        return warp_total(total);
    }

    // The first id, in ascending order, at which the sum of weight(z, id) passes `target`; `mine` is the sum over
    // this warp's stretch of the slice (warps take consecutive stretches).  -1 in CTAs that do not hold it.
    __device__ __forceinline__ int warp_stretch() const { return (vectors + kSampleWarps - 1) / kSampleWarps; }
    // This warp's part of the sum of weights that are kept.
    __device__ __forceinline__ uint64_t kept_sum(const Kept &kept) {
        const int n = warp_stretch(), from = static_cast<int>(threadIdx.x >> 5) * n, to = min(from + n, vectors);
        const int lane = static_cast<int>(threadIdx.x & 31);
        uint64_t s = 0;
        auto add = [&](float, uint64_t weight, uint32_t) { s += weight; };
        if (every(kept)) {
            weigh_all(from, to, 32, lane, add);
        } else {
            const Bounds bounds(kept);
            scan(from, to, 32, lane, kept.border(), [&](const uint4 &w, int v, bool) {
                weigh_vector(w, v, [&](const float(&z)[kVec], int first) { return bounds.mask(z, first); }, add);
            });
        }
        return s;
    }
    // This warp's part of the tokens that pred takes.
    template <class Pred>
    __device__ __forceinline__ uint64_t count_sum(float border, Pred &&pred) {
        const int n = warp_stretch(), from = static_cast<int>(threadIdx.x >> 5) * n, to = min(from + n, vectors);
        uint64_t s = 0;
        scan(from, to, 32, static_cast<int>(threadIdx.x & 31), border, [&](const uint4 &w, int v, bool in) {
            float z[kVec];
            decode_vec<D>(w, z);
#pragma unroll
            for (int e = 0; e < kVec; ++e) {
                const int id = first_id + v * kVec + e;
                s += in && id < P.V && pred(z[e], id) ? 1 : 0;
            }
        });
        return s;
    }
    // Whether no token is left out.
    __device__ __forceinline__ bool every(const Kept &kept) const { return kept.border() == -INFINITY && kept.id >= P.V; }
    // Publishes the stretches' sums; returns the cluster's total, and what lies before this CTA in `before`.
    __device__ __forceinline__ uint64_t publish(uint64_t s, uint64_t &before) {
        s = warp_total(s);
        if ((threadIdx.x & 31) == 0) S.stretches[threadIdx.x >> 5] = s;
        const uint64_t x = exchange([&] {
            uint64_t all = 0;
#pragma unroll
            for (int w = 0; w < kSampleWarps; ++w) all += S.stretches[w];
            return all;
        });
        before = warp_total(static_cast<int>(threadIdx.x & 31) < rank ? x : 0);
        return warp_total(x);
    }
    // The CTA that holds the target takes the warp's stretch that does, a vector to a thread.  The warp that finds the
    // token returns its id, every other -1.
    template <class Weight>
    __device__ __forceinline__ int locate(Weight &&weight, uint64_t before, uint64_t target, float &value) {
        int w = 0;
        uint64_t run = before;
        for (; w < kSampleWarps; ++w) {
            const uint64_t s = S.stretches[w];
            if (run <= target && run + s > target) break;
            run += s;
        }
        if (w == kSampleWarps) return -1;
        const int t = static_cast<int>(threadIdx.x), lane = t & 31;
        const int n = warp_stretch(), v = w * n + t, to = min((w + 1) * n, vectors);
        float z[kVec];
        uint64_t upto = 0, x = 0;
        if (w * n + (t & ~31) < to) {  // whole warps
            decode_vec<D>(vector(v, to), z);
#pragma unroll
            for (int e = 0; e < kVec; ++e) {
                const int id = first_id + v * kVec + e;
                x += weight(z[e], id, v < to && id < P.V);
            }
            upto = x;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const uint64_t y = __shfl_up_sync(kAll, upto, o);
                if (lane >= o) upto += y;
            }
        }
        if (lane == 31) S.red[t >> 5] = upto;
        __syncthreads();
        for (int i = 0; i < (t >> 5); ++i) run += S.red[i];
        const uint32_t over = __ballot_sync(kAll, run + upto > target && run + upto - x <= target);
        if (!over) return -1;
        int id = -1;
        float at = 0.f;
        x = run + upto - x;
#pragma unroll
        for (int e = 0; e < kVec; ++e) {
            x += weight(z[e], first_id + v * kVec + e, v < to && first_id + v * kVec + e < P.V);
            if (id < 0 && x > target) id = first_id + v * kVec + e, at = z[e];
        }
        const int l = __ffs(over) - 1;
        value = __shfl_sync(kAll, at, l);
        return __shfl_sync(kAll, id, l);
    }

    // The weight of a token that is in; all lanes of a warp call, and skip it together where none is.
    __device__ __forceinline__ uint64_t weight_if(float z, bool in) {
        in = in && z > -INFINITY;
        if (!__any_sync(kAll, in)) return 0;
        const uint64_t x = weigh(in ? z : m);
        return in ? x : 0;
    }

    // The first histogram: `shift` bits of d to a range from `near` on, what is nearer and what is farther in one range
    // each.
    struct First {
        uint32_t near = kNear, shift = kFirstShift;
        __device__ __forceinline__ int bin(uint32_t d) const {
            return min(max((static_cast<int>(d - near) >> shift) + 1, 0), kBins - 1);
        }
        __device__ __forceinline__ uint32_t start(uint32_t bin) const {  // `near` may lie below 0
            return bin == 0 ? 0 : static_cast<uint32_t>(max(static_cast<int>(near + ((bin - 1) << shift)), 0));
        }
        __device__ __forceinline__ uint32_t end(uint32_t bin) const { return bin == kBins - 1 ? kInfinite + 1 : near + (bin << shift); }
    };
    // A range of d, from 0 on, that holds the largest tokens of at least k threads (k at most the cluster's threads).
    __device__ __forceinline__ uint32_t range_of_top(int k) {
        Histogram &H = S.hist[1];
        const int t = static_cast<int>(threadIdx.x);
        H.count[t] = 0;
        __syncthreads();
        const First F;
        atomicAdd(&H.count[F.bin(distance(top))], 1u);
        cluster.sync();
        uint32_t count = 0;
#pragma unroll 8
        for (int c = 0; c < ctas; ++c) count += cluster.map_shared_rank(&H, c)->count[t];
        uint32_t upto = count;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const uint32_t x = __shfl_up_sync(kAll, upto, o);
            if ((t & 31) >= o) upto += x;
        }
        if ((t & 31) == 31) S.red[t >> 5] = upto;
        __syncthreads();
        for (int w = 0; w < (t >> 5); ++w) upto += static_cast<uint32_t>(S.red[w]);
        if (upto - count < static_cast<uint32_t>(k) && upto >= static_cast<uint32_t>(k)) S.found_bin = static_cast<uint32_t>(t);
        __syncthreads();
        return F.end(S.found_bin);
    }

    // Narrows `kept` to the ranks that a limit leaves.  kMass: while the weight above a rank is below `share` of
    // what is kept; else the first `k` ranks.
    template <bool kMass>
    __device__ void limit_to(Kept &kept, int k, float share) {
        uint32_t lo = 0, hi = kInfinite + 1, shift = 0;  // bits of d: the range looked at
        bool first = true;
        uint64_t above = 0, in_range = 0;  // tokens or weight above the range; tokens in it
        uint64_t goal = static_cast<uint64_t>(k);
        float border = -INFINITY;
        First F;
        bool few = false;  // the range may hold at most kList tokens
        uint32_t light = 0xFFFFFFFFu;  // d from which tokens only count for the total
        if (kMass) {
            border = kept.border();
            // What lies beyond tau ln(V / (1 - share)) weighs less than 1 - share of the largest alone, so the border
            // comes before it.  (Beyond the histogram's evenly divided part nothing is left out.)
            const float d = 1.0001f / weigh.c_hi * log2f(static_cast<float>(P.V) / (1.f - share));
            if (d < 1000.f) {
                light = __float_as_uint(d);
                // 128 ranges for each power of two up to there: the tokens are many where the distances are large, and
                // atomics on one range wait for one another
                F.shift = kFirstShift - 2;
                F.near = light - ((kBins - 2) << F.shift);
            }
        } else if (k <= ctas * kSampleThreads) {
            // k threads' largest tokens are k tokens: no token beyond the k-th of those is among the k first
            hi = range_of_top(k);
            border = nearest(hi);
            few = k <= kList / 2;
        }
        uint32_t low_key = 0xFFFFFFFFu, high_key = 0;  // the smallest and the largest value of the range
        auto look_at_values = [&]() {
            low_key = 0xFFFFFFFFu, high_key = 0;
            each(nearest(hi), [&](float z, int id, bool there) {
                const uint32_t d = distance(z);
                if (there && d >= lo && d < hi && (!kMass || kept(z, id))) {
                    const uint32_t o = ordered_bits(z);
                    low_key = min(low_key, o), high_key = max(high_key, o);
                }
            });
            low_key = __reduce_min_sync(kAll, low_key), high_key = __reduce_max_sync(kAll, high_key);
            if ((threadIdx.x & 31) == 0) S.sums[turn][0][threadIdx.x >> 5] = low_key, S.sums[turn][1][threadIdx.x >> 5] = high_key;
            cluster.sync();
            gather(&S.sums[turn][0][0], [&](int, uint64_t x) { low_key = min(low_key, static_cast<uint32_t>(x)); });
            gather(&S.sums[turn][1][0], [&](int, uint64_t x) { high_key = max(high_key, static_cast<uint32_t>(x)); });
            low_key = __reduce_min_sync(kAll, low_key), high_key = __reduce_max_sync(kAll, high_key);
            turn ^= 1;
        };
        // a level divides its range by 512: three and the first end at single distances
        for (int level = 0; level < 8; ++level) {
            if (few && rank_range<kMass>(kept, lo, hi, above, goal)) return;
            // Many tokens of a narrow range: of one value as a rule (a bf16 row has few), which rank by id.
            if (level >= 2 || (!first && hi - lo == 1)) {
                look_at_values();
                if (low_key == high_key || hi - lo == 1) break;
            }
            Histogram &H = S.hist[level & 1];
            const int t = static_cast<int>(threadIdx.x);
            H.count[t] = 0;
            if (kMass) H.mass[t] = make_uint2(0, 0);
            __syncthreads();
            uint64_t rest = 0;
            auto add = [&](int bin, uint64_t w) {
                const uint32_t part = static_cast<uint32_t>(w);
                const uint32_t was = atomicAdd(&H.mass[bin].x, part);
                const uint32_t carry = was + part < was ? 1u : 0u;
                const uint32_t more = static_cast<uint32_t>(w >> 32) + carry;
                if (more) atomicAdd(&H.mass[bin].y, more);
            };
            auto bin_of = [&](uint32_t d) { return first ? F.bin(d) : static_cast<int>((d - lo) >> shift); };
            const float from = first ? border : nearest(hi);
            if (kMass) {
                auto put = [&](float z, uint64_t weight, uint32_t times) {
                    const uint32_t d = distance(z);
                    if (d >= min(light, kInfinite)) {
                        rest += weight;
                    } else {
                        add(bin_of(d), weight);
                        atomicAdd(&H.count[bin_of(d)], times);
                    }
                };
                if (first && every(kept)) {
                    weigh_all(0, vectors, kSampleThreads, t, put);
                } else {
                    const Bounds bounds(kept);
                    scan(0, vectors, kSampleThreads, t, from, [&](const uint4 &w, int v, bool) {
                        weigh_vector(
                            w, v,
                            [&](const float(&z)[kVec], int first_of) {
                                uint32_t mask = bounds.mask(z, first_of);
#pragma unroll
                                for (int e = 0; e < kVec; ++e)
                                    if (distance(z[e]) - lo >= hi - lo) mask &= ~(1u << e);
                                return mask;
                            },
                            put);
                    });
                }
            } else {
                // what lies beyond the row counts as -inf, and ranks behind the row's own by its ids
                scan(0, vectors, kSampleThreads, t, from, [&](const uint4 &w, int, bool) {
                    float z[kVec];
                    decode_vec<D>(w, z);
                    const bool flat = alike(w);  // constant rows
#pragma unroll
                    for (int e = 0; e < kVec; ++e) {
                        const uint32_t d = distance(z[e]);
                        if (d - lo < hi - lo && (!flat || (t & 31) == 0)) atomicAdd(&H.count[bin_of(d)], flat ? 32u : 1u);
                    }
                });
            }
            if (kMass && first && light != 0xFFFFFFFFu) {
                rest = warp_total(rest);
                if ((t & 31) == 0 && rest) add(kBins - 1, rest);
            }
            cluster.sync();
            // every CTA adds up all histograms: thread t bin t
            uint32_t count = 0;
            uint64_t mass = 0;
#pragma unroll 8
            for (int c = 0; c < ctas; ++c) {
                const Histogram *h = cluster.map_shared_rank(&H, c);
                count += h->count[t];
                if (kMass) {
                    const uint2 w = h->mass[t];
                    mass += (static_cast<uint64_t>(w.y) << 32) + w.x;
                }
            }
            const uint64_t mine = kMass ? mass : count;
            uint64_t upto = mine;
            const int lane = t & 31;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const uint64_t x = __shfl_up_sync(kAll, upto, o);
                if (lane >= o) upto += x;
            }
            if (lane == 31) S.red[t >> 5] = upto;
            __syncthreads();
            uint64_t before = 0, total = 0;
            for (int w = 0; w < kSampleWarps; ++w) {
                const uint64_t x = S.red[w];
                if (w < (t >> 5)) before += x;
                total += x;
            }
            upto += before;
            if (kMass && first) {
                // sums are whole numbers: below share * total is below that rounded up
                if (t == 0) S.goal = static_cast<uint64_t>(ceil(static_cast<double>(share) * static_cast<double>(total)));
                __syncthreads();
                goal = S.goal;
            }
            if (mine && above + upto - mine < goal && above + upto >= goal) {
                S.found_bin = static_cast<uint32_t>(t);
                S.found_above = above + upto - mine;
                S.found_in = count;
            }
            __syncthreads();
            const uint32_t bin = S.found_bin;
            above = S.found_above;
            in_range = S.found_in;
            if (first) {
                lo = F.start(bin);
                hi = min(min(hi, F.end(bin)), light);
                first = false;
                light = 0xFFFFFFFFu;
            } else {
                lo += bin << shift;
                hi = min(hi, lo + (1u << shift));
            }
            few = in_range <= kList;
            shift = 0;
            while (((hi - lo - 1) >> shift) >= kBins) ++shift;
            __syncthreads();
        }
        // Distances are rounded, so values far below the largest may share one: then the last value kept is found bit by
        // bit.
        const int t = static_cast<int>(threadIdx.x);
        uint32_t key = low_key;
        if (low_key != high_key) {
            key = 0;
            auto upto = [&](uint32_t from) {  // tokens or weight of the range from that key on
                uint64_t s = 0;
                each(nearest(hi), [&](float z, int id, bool there) {
                    const uint32_t d = distance(z);
                    const bool in = there && d >= lo && d < hi && ordered_bits(z) >= from && (!kMass || kept(z, id));
                    s += kMass ? weight_if(z, in) : static_cast<uint64_t>(in);
                });
                return cluster_sum(s);
            };
            for (int bit = 31; bit >= 0; --bit) {
                const uint32_t c = key | (1u << bit);
                if (c <= high_key && above + upto(c) >= goal) key = c;
            }
            if (key < 0xFFFFFFFFu) above += upto(key + 1);
        }
        // ranks of that value: kept while what is above them is below the goal
        const float value = value_of_ordered(key);
        uint64_t ties = goal - above;
        if (kMass) {
            const uint64_t one = weigh(value);
            ties = one ? (goal - above + one - 1) / one : 1;
        }
        auto is_tie = [&](float z, int id) { return z == value && (!kMass || kept(z, id)); };
        auto tie = [&](float z, int id, bool there) { return static_cast<uint64_t>(there && is_tie(z, id)); };
        uint64_t before;
        publish(count_sum(value, is_tie), before);
        float unused;
        const int id = locate(tie, before, ties - 1, unused);
        if (id >= 0 && (t & 31) == 0)
            for (int c = 0; c < ctas; ++c) *cluster.map_shared_rank(&S.result, c) = id;
        cluster.sync();
        kept.last = value;
        kept.id = S.result;
    }

    // The tokens with lo <= d < hi against one another; false, and nothing done, if they are more than kList.
    template <bool kMass>
    __device__ __forceinline__ bool rank_range(Kept &kept, uint32_t lo, uint32_t hi, uint64_t above, uint64_t goal) {
        const int t = static_cast<int>(threadIdx.x);
        if (t == 0) S.listed = 0;
        __syncthreads();
        each(nearest(hi), [&](float z, int id, bool there) {
            const uint32_t d = distance(z);
            if (there && d >= lo && d < hi && (!kMass || kept(z, id))) {
                const int at = atomicAdd(&S.listed, 1);
                if (at < kList) S.list[at] = make_key(z, id);
            }
        });
        // how many each CTA has, and how many the CTAs before it
        const uint32_t here = static_cast<uint32_t>(exchange([&] { return static_cast<uint64_t>(S.listed); }));
        uint32_t upto = here;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const uint32_t x = __shfl_up_sync(kAll, upto, o);
            if ((t & 31) >= o) upto += x;
        }
        const int n = static_cast<int>(__shfl_sync(kAll, upto, 31));
        if (n > kList) return false;
        int cta = 0;  // that holds number t
        for (int c = 0; c < ctas; ++c) cta += t >= static_cast<int>(__shfl_sync(kAll, upto, c)) ? 1 : 0;
        const int at = t - static_cast<int>(__shfl_sync(kAll, upto - here, cta & 31));
        if (t < n) S.ranked[t] = cluster.map_shared_rank(&S.list[0], cta)[at];
        __syncthreads();
        const uint64_t own = t < n ? S.ranked[t] : 0;
        if (kMass && t < kList) {
            const uint64_t w = weight_if(key_value(own), t < n);
            S.ranked_weight[t] = w;
        }
        __syncthreads();
        bool in = false;
        int place = 0;
        if (t < n) {
            uint64_t higher = above;
            for (int i = 0; i < n; ++i)
                if (S.ranked[i] > own) {
                    ++place;
                    if (kMass) higher += S.ranked_weight[i];
                }
            if (!kMass) higher += static_cast<uint64_t>(place);
            in = higher < goal;
        }
        const int left = __syncthreads_count(in);
        if (in && place == left - 1) S.found_above = own;
        __syncthreads();
        const uint64_t last = S.found_above;
        kept.last = key_value(last);
        kept.id = key_id(last);
        // the next limit's histogram may use what others still read: they are past it after its own barrier
        return true;
    }
};

template <class D>
__global__ void __launch_bounds__(kSampleThreads) sample_kernel(const __grid_constant__ SampleParams P) {
    extern __shared__ __align__(16) uint8_t raw[];
    Shared &S = *reinterpret_cast<Shared *>(raw);
    uint4 *slice = reinterpret_cast<uint4 *>(raw + (sizeof(Shared) + 15) / 16 * 16);
    constexpr int kVec = D::kVec;
    Row<D> R(P, S, slice);
    asm volatile("barrier.cluster.arrive;" ::: "memory");
    const int row = static_cast<int>(blockIdx.x) / R.ctas, tid = threadIdx.x, lane = tid & 31;
    const int64_t at = static_cast<int64_t>(row) * P.ld;

    // ---- the slice, its largest logit (lowest id) and its validity --------------------------
    uint64_t best = 0;
    int odd = 0;
    const char *src = static_cast<const char *>(P.logits) + (at + R.first_id) * D::kBytes;
    float top = -INFINITY;
    int top_at = -1;
    auto look = [&](int v, const uint4 &w) {  // a thread's vectors come in ascending order
        const float x = vector_max<D>(w);
        odd |= vector_nan<D>(w);
        if (x > top) top = x, top_at = v;
    };
    const int whole = P.aligned ? max(0, min(R.vectors, (P.V - R.first_id) / kVec)) : 0;
    constexpr int kFlight = 4;
    for (int v0 = tid; v0 < whole; v0 += kSampleThreads * kFlight) {
        uint4 w[kFlight];
#pragma unroll
        for (int i = 0; i < kFlight; ++i) {
            const int v = v0 + i * kSampleThreads;
            if (v < whole) w[i] = __ldcs(reinterpret_cast<const uint4 *>(src) + v);
        }
#pragma unroll
        for (int i = 0; i < kFlight; ++i) {
            const int v = v0 + i * kSampleThreads;
            if (v < whole) {
                slice[v] = w[i];
                look(v, w[i]);
            }
        }
    }
    for (int v = whole + tid; v < R.vectors; v += kSampleThreads) {
        float z[kVec];
#pragma unroll
        for (int e = 0; e < kVec; ++e) {
            const int id = R.first_id + v * kVec + e;
            z[e] = id < P.V ? load_logit<D>(P.logits, at + id) : -INFINITY;
        }
        uint4 w;
        uint32_t *words = &w.x;
#pragma unroll
        for (int e = 0; e < 4; ++e)
            words[e] = kVec == 4 ? __float_as_uint(z[e])
                                 : (__float_as_uint(z[2 * e % kVec]) >> 16) | (__float_as_uint(z[(2 * e + 1) % kVec]) & 0xFFFF0000u);
        slice[v] = w;
        look(v, w);
    }
    odd |= top == INFINITY;
    if (top_at >= 0) {
        float z[kVec];
        decode_vec<D>(slice[top_at], z);
#pragma unroll
        for (int e = kVec - 1; e >= 0; --e)
            if (z[e] == top) best = make_key(top, R.first_id + top_at * kVec + e);
    }
    constexpr uint64_t kOdd = ~0ull;  // no token's key
    if (odd) best = kOdd;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        const uint64_t t = __shfl_xor_sync(kAll, best, o);
        best = t > best ? t : best;
    }
    if (lane == 0) S.best[tid >> 5] = best;
    if (tid == kSampleThreads - 1 && P.min_p) {
        // 64-bit arithmetic is slow here: one thread does it
        const float least = P.min_p[row];
        if (least > 0.f) S.drop = static_cast<double>(P.tau[row]) * log(static_cast<double>(least));
    }
    asm volatile("barrier.cluster.wait;" ::: "memory");  // every CTA has started: it can be written to
    best = R.exchange([&] {
        uint64_t most = 0;
#pragma unroll
        for (int w = 0; w < kSampleWarps; ++w) most = S.best[w] > most ? S.best[w] : most;
        return most;
    });
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        const uint64_t t = __shfl_xor_sync(kAll, best, o);
        best = t > best ? t : best;
    }
    odd = best == kOdd;
    const float m = best && !odd ? key_value(best) : -INFINITY;
    const float tau = P.tau[row], u = P.u[row];
    const int top_k = P.top_k ? P.top_k[row] : 0;
    const float top_p = P.top_p ? P.top_p[row] : 1.f;
    const float min_p = P.min_p ? P.min_p[row] : 0.f;
    int bad = 0;
    if (odd || !(m > -INFINITY)) bad |= SSD_DEV_NONFINITE;
    if (!(tau >= 0.f) || !(tau < INFINITY)) bad |= SSD_DEV_BAD_TEMPERATURE;
    if (top_p != top_p || min_p != min_p || !(u >= 0.f && u < 1.f)) bad |= SSD_DEV_BAD_PARAM;

    const Kept only{m, key_id(best), -INFINITY};
    Kept kept{-INFINITY, P.V, -INFINITY};
    if (bad) {
        if (R.rank == 0 && tid == 0) {
            report(P.dev_status, bad);
            P.tokens[row] = -1;
            if (P.prob) P.prob[row] = __int_as_float(0x7FC00000);
        }
    } else if (tau == 0.f) {
        kept = only;
        if (R.rank == 0 && tid == 0) {
            P.tokens[row] = only.id;
            if (P.prob) P.prob[row] = 1.f;
        }
    } else {
        R.m = m;
        R.top = top;
        R.weigh.m = m;
        // log2(e) / tau as two floats: the quotient, and what it left over
        constexpr float kLog2eHigh = 1.44269502f, kLog2eLow = 1.92596299e-8f;
        const float c = __fdiv_rn(kLog2eHigh, tau);
        R.weigh.c_hi = fminf(c, 1e30f);
        R.weigh.c_lo = c < 1e30f ? __fdiv_rn(fmaf(-c, tau, kLog2eHigh) + kLog2eLow, tau) : 0.f;
        R.weigh.table = __ldg(&kPowers[lane]);
        if (top_k > 0 && top_k < P.V) R.template limit_to<false>(kept, top_k, 0.f);
        if (top_p <= 0.f || min_p > 1.f)
            kept = only;
        else if (top_p < 1.f)
            R.template limit_to<true>(kept, 0, top_p);
        // w >= min_p as a least logit, rounded up to a float; the largest logit stays
        if (min_p > 0.f) kept.least = min_p >= 1.f ? m : __double2float_ru(static_cast<double>(m) + S.drop);
        // ---- the first id at which the kept weight passes u of its total ------------------------
        const bool all = R.every(kept);
        auto weight = [&](float z, int id, bool there) { return R.weight_if(z, there && (all || kept(z, id))); };
        uint64_t before;
        const uint64_t total = R.publish(R.kept_sum(kept), before);
        if (tid == 0) S.target = static_cast<uint64_t>(static_cast<double>(u) * static_cast<double>(total));
        __syncthreads();
        float z;
        const int token = R.locate(weight, before, S.target, z);
        if (token >= 0) {
            uint32_t value;
            int shift;
            R.weigh.parts(z, value, shift);
            if (lane == 0) {
                P.tokens[row] = token;
                // value * 2^-(27 + shift) of total * 2^-43
                if (P.prob)
                    P.prob[row] = static_cast<float>(static_cast<double>(value) * __hiloint2double((1023 + 16 - shift) << 20, 0) /
                                                     static_cast<double>(total));
            }
        }
    }
    if (P.filtered) {
        const uint32_t dropped = kVec == 4 ? __float_as_uint(SSD_DROPPED_LOGIT)
                                           : static_cast<uint32_t>(__bfloat16_as_ushort(__float2bfloat16(SSD_DROPPED_LOGIT)));
        // e^-104 is 0 in fp32: next to a largest logit that is 104 tau above it, a dropped token weighs nothing.  A row that
        // lies lower is left as it is, and reported if a token of it had to be dropped.  (Temperatures count up to 900,
        // where that is 93600 and any row from -6000 on fits.)
        const bool low = !bad && !(m - __uint_as_float(kVec == 4 ? dropped : dropped << 16) > 104.f * fminf(tau, 900.f));
        bool kept_back = false;
        for (int v = tid; v < R.vectors; v += kSampleThreads) {
            uint4 w = slice[v];
            uint32_t *words = &w.x;
            if (!bad) {
                float z[kVec];
                decode_vec<D>(w, z);
#pragma unroll
                for (int e = 0; e < kVec; ++e) {
                    if (kept(z[e], R.first_id + v * kVec + e) && z[e] > -INFINITY) continue;
                    if (low) {
                        kept_back |= R.first_id + v * kVec + e < P.V;
                        continue;
                    }
                    if (kVec == 4)
                        words[e % 4] = dropped;
                    else
                        words[e / 2 % 4] = e % 2 ? (words[e / 2 % 4] & 0xFFFFu) | (dropped << 16) : (words[e / 2 % 4] & 0xFFFF0000u) | dropped;
                }
            }
            if (v < whole) {
                __stcs(reinterpret_cast<uint4 *>(static_cast<char *>(P.filtered) + (at + R.first_id) * D::kBytes) + v, w);
            } else {
                float z[kVec];
                decode_vec<D>(w, z);
#pragma unroll
                for (int e = 0; e < kVec; ++e) {
                    const int id = R.first_id + v * kVec + e;
                    if (id < P.V) store_logit<D>(P.filtered, at + id, z[e]);
                }
            }
        }
        if (kept_back) report(P.dev_status, SSD_DEV_LOW_LOGITS);
    }
}

constexpr size_t kFixedBytes = (sizeof(Shared) + 15) / 16 * 16;

template <class D>
int sample_launch(SampleParams P, cudaStream_t stream) {
    int dev = 0, sms = 0, most = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&most, cudaDevAttrMaxSharedMemoryPerBlockOptin, dev) != cudaSuccess) {
        cudaGetLastError();
        return SSD_ERR_CUDA;
    }
    auto *kernel = sample_kernel<D>;
    static std::atomic<uint64_t> ready{0};
    const uint64_t bit = 1ull << (dev & 63);
    if (!(ready.load(std::memory_order_relaxed) & bit)) {
        if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, most) != cudaSuccess ||
            cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) != cudaSuccess) {
            cudaGetLastError();
            return SSD_ERR_CUDA;
        }
        ready.fetch_or(bit, std::memory_order_relaxed);
    }
    // The fewest CTAs to a row that leave two of them on an SM; more, down to 4 KB slices, where the rows are too
    // few to fill the GPU.
    const int vectors = (P.V + D::kVec - 1) / D::kVec;
    auto slice = [&](int ctas) { return (vectors + ctas - 1) / ctas; };
    int ctas = 1;
    while (ctas < 16 && kFixedBytes + static_cast<size_t>(slice(ctas)) * 16 > 112 * 1024) ctas *= 2;
    while (ctas < 16 && static_cast<int64_t>(P.rows) * ctas * 2 <= 2 * sms && slice(ctas * 2) >= 256) ctas *= 2;
    P.slice = slice(ctas);
    const size_t dyn = kFixedBytes + static_cast<size_t>(P.slice) * 16;
    if (dyn > static_cast<size_t>(most) || static_cast<int64_t>(P.rows) * ctas > 0x7FFFFFFF) return SSD_ERR_UNSUPPORTED;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(P.rows * ctas));
    cfg.blockDim = dim3(kSampleThreads);
    cfg.dynamicSmemBytes = dyn;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = static_cast<unsigned>(ctas);
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (cudaLaunchKernelEx(&cfg, kernel, P) != cudaSuccess) {
        cudaGetLastError();
        return SSD_ERR_CUDA;
    }
    return SSD_OK;
}

}  // namespace
}  // namespace ssd

extern "C" int ssd_sample(const void *logits, int dtype, int rows, int V, int64_t ld, const float *temperature,
                          const int32_t *top_k, const float *top_p, const float *min_p, const float *uniforms,
                          int32_t *tokens, float *prob, void *filtered, int32_t *dev_status, void *stream) {
    using namespace ssd;
    if (dtype != SSD_F32 && dtype != SSD_BF16) return SSD_ERR_DTYPE;
    if (!logits || !temperature || !uniforms || !tokens || rows < 1 || V < 2 || ld < V) return SSD_ERR_INVALID_ARG;
    if (V > (dtype == SSD_F32 ? SSD_MAX_V_F32 : SSD_MAX_V_BF16)) return SSD_ERR_UNSUPPORTED;
    const int bytes = dtype == SSD_F32 ? 4 : 2;
    SampleParams P{logits,   rows,   V,    ld,       temperature, top_k, top_p, min_p,
                   uniforms, tokens, prob, filtered, dev_status,  0,     0};
    P.aligned = aligned(logits, 16) && (rows == 1 || ld * bytes % 16 == 0) && (!filtered || aligned(filtered, 16));
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    return dtype == SSD_F32 ? sample_launch<F32Tag>(P, s) : sample_launch<BF16Tag>(P, s);
}
