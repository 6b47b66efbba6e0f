// ssd_sample.cu -- one token per logit row under temperature, top-k, top-p and min-p
// (sm_103a).
//
// What is kept is a prefix of the ranking (logit desc, id asc), so it is described by its
// last value and, among tokens of that value, its last id.  Each limit is found bit by
// bit on the ordered bits of the logit with counts (top-k) or sums of weights (top-p).
//
// Weights.  w = exp((z - m) / tau) = 2^t, t = d * c with d = z - m and c = log2(e) / tau
// both carried as two floats, so that t is exact to about 2^-45 of itself.  t is split
// into k / 32 + g: a 32-entry table of 2^(i/32) (one entry per lane, read by shuffle) times
// a polynomial of 2^g - 1, |g| <= 1/64, gives 28 significant bits, which are shifted into
// 64-bit fixed point with 43 bits after the point.  Sums of those are exact: they depend
// on no order, a prefix and a total agree to the last bit, and the rank or id at which a
// sum passes its limit is decided as the real numbers would, but for cases closer than
// 2^-28 of a weight.
//
// One CTA per row; every pass reads the row again (L2 holds it).
#include <cuda_bf16.h>

#include "ssd_kv.h"
#include "ssd_device.cuh"

namespace ssd {
namespace {

constexpr int kSampleThreads = 1024;
constexpr int kSampleWarps = kSampleThreads / 32;

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
};

// 2^t in fixed point, t = (z - m) * (c_hi + c_lo) <= 0.  All lanes call; `table` is this
// lane's 2^(lane/32) in units of 2^-27.
struct Weigher {
    float m, c_hi, c_lo;
    uint32_t table;
    __device__ __forceinline__ uint64_t operator()(float z) const {
        const float d = z - m;
        // what the subtraction rounded off, exact (m >= z; both finite)
        const float bb = d - z;
        const float err = (z - (d - bb)) + (-m - bb);
        float t = d * c_hi;
        const float t_lo = fmaf(d, c_lo, fmaf(d, c_hi, -t)) + err * c_hi;
        t = fmaxf(t, -64.f);
        const float magic = 12582912.f;  // 1.5 * 2^23: the sum's low bits are the rounded value
        const float km = fmaf(t, 32.f, magic);
        const int k = __float_as_int(km) - __float_as_int(magic);
        const float g = fmaf(km - magic, -0.03125f, t) + t_lo;
        // (2^g - 1) = g (ln2 + g (ln2^2/2 + g (ln2^3/6 + g ln2^4/24)))
        float q = fmaf(g, 0.0096181291f, 0.0555041087f);
        q = fmaf(g, q, 0.2402265070f);
        q = fmaf(g, q, 0.6931471806f) * g;
        const uint32_t base = __shfl_sync(0xFFFFFFFFu, table, k & 31);
        const int more = __float_as_int(fmaf(static_cast<float>(base), q, magic)) - __float_as_int(magic);
        const uint64_t v = static_cast<uint64_t>(base + static_cast<uint32_t>(more)) << 16;
        const int shift = -(k >> 5);
        return t > -60.f ? v >> shift : 0;
    }
};

template <class T>
__device__ __forceinline__ T sample_sum(T v, T *red) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
    __syncthreads();
    T r = 0;
    for (int w = 0; w < kSampleWarps; ++w) r += red[w];
    return r;
}

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

// What is kept: ordered value above `key`, or equal to it and id <= `id`; and value >= `least`.
struct Kept {
    uint32_t key;
    int id;
    float least;
    __device__ __forceinline__ bool operator()(float z, int i) const {
        const uint32_t o = ordered_bits(z);
        return (o > key || (o == key && i <= id)) && z >= least;
    }
};

template <class D>
__global__ void __launch_bounds__(kSampleThreads) sample_kernel(const __grid_constant__ SampleParams P) {
    __shared__ uint64_t red[kSampleWarps];
    __shared__ uint64_t scan[kSampleThreads];
    __shared__ int red_i[kSampleWarps];
    __shared__ uint64_t hit_before;
    __shared__ int hit_thread;
    const int row = blockIdx.x, tid = threadIdx.x, lane = tid & 31;
    const int V = P.V;
    const int64_t at = static_cast<int64_t>(row) * P.ld;
    // V rounded up so that whole warps call the weigher
    const int V32 = (V + 31) & ~31;

    // largest logit (lowest id), and the row's validity
    uint64_t best = 0;
    int odd = 0;
    for (int i = tid; i < V; i += kSampleThreads) {
        const float z = load_logit<D>(P.logits, at + i);
        odd |= !(z < INFINITY);
        const uint64_t k = make_key(z, i);
        best = k > best ? k : best;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        const uint64_t t = __shfl_xor_sync(0xFFFFFFFFu, best, o);
        best = t > best ? t : best;
    }
    if (lane == 0) red[tid >> 5] = best;
    odd = __syncthreads_or(odd);
    for (int w = 0; w < kSampleWarps; ++w) best = red[w] > best ? red[w] : best;
    const float m = key_value(best);
    const float tau = P.tau[row], u = P.u[row];
    const int top_k = P.top_k ? P.top_k[row] : 0;
    const float top_p = P.top_p ? P.top_p[row] : 1.f;
    const float min_p = P.min_p ? P.min_p[row] : 0.f;
    int bad = 0;
    if (odd || !(m > -INFINITY)) bad |= SSD_DEV_NONFINITE;
    if (!(tau >= 0.f) || !(tau < INFINITY)) bad |= SSD_DEV_BAD_TEMPERATURE;
    if (top_p != top_p || min_p != min_p || !(u >= 0.f && u < 1.f)) bad |= SSD_DEV_BAD_PARAM;
    if (bad) {
        if (tid == 0) {
            report(P.dev_status, bad);
            P.tokens[row] = -1;
            if (P.prob) P.prob[row] = __int_as_float(0x7FC00000);
        }
        if (P.filtered)
            for (int i = tid; i < V; i += kSampleThreads)
                store_logit<D>(P.filtered, at + i, load_logit<D>(P.logits, at + i));
        return;
    }

    Kept kept{0u, V, -INFINITY};
    int token = key_id(best);
    float prob = 1.f;
    if (tau == 0.f) {
        kept = Kept{static_cast<uint32_t>(best >> 32), token, -INFINITY};
    } else {
        const double c = fmin(1.4426950408889634074 / static_cast<double>(tau), 1e30);
        Weigher w;
        w.m = m;
        w.c_hi = static_cast<float>(c);
        w.c_lo = static_cast<float>(c - static_cast<double>(w.c_hi));
        w.table = static_cast<uint32_t>(rint(exp2(static_cast<double>(lane) / 32.0) * 134217728.0));

        auto count = [&](auto &&pred) {
            int n = 0;
            for (int i = tid; i < V; i += kSampleThreads) n += pred(load_logit<D>(P.logits, at + i), i) ? 1 : 0;
            return sample_sum(n, red_i);
        };
        auto mass = [&](auto &&pred) {
            uint64_t s = 0;
            for (int i = tid; i < V32; i += kSampleThreads) {
                const float z = i < V ? load_logit<D>(P.logits, at + i) : -INFINITY;
                const bool in = i < V && z > -INFINITY && pred(z, i);
                const uint64_t x = w(in ? z : m);
                s += in ? x : 0;
            }
            return sample_sum(s, red);
        };
        if (top_k > 0 && top_k < V) {
            // the value of rank top_k: the largest that at least top_k tokens reach
            uint32_t key = 0;
            for (int bit = 31; bit >= 0; --bit) {
                const uint32_t c2 = key | (1u << bit);
                if (count([&](float z, int) { return ordered_bits(z) >= c2; }) >= top_k) key = c2;
            }
            const int above = count([&](float z, int) { return ordered_bits(z) > key; });
            // among tokens of that value, the lowest ids
            int id = 0;
            for (int bit = 30; bit >= 0; --bit) {
                const int c2 = id + (1 << bit);
                if (c2 < V &&
                    count([&](float z, int i) { return ordered_bits(z) == key && i < c2; }) < top_k - above)
                    id = c2;
            }
            kept.key = key, kept.id = id;
        }
        if (top_p < 1.f) {
            const uint64_t total = mass(kept);
            const double limit = static_cast<double>(top_p) * static_cast<double>(total);
            // the last value kept: the largest v such that the values >= v hold the limit
            uint32_t key = 0;
            for (int bit = 31; bit >= 0; --bit) {
                const uint32_t c2 = key | (1u << bit);
                const uint64_t s = mass([&](float z, int i) { return kept(z, i) && ordered_bits(z) >= c2; });
                if (static_cast<double>(s) >= limit && s > 0) key = c2;
            }
            const uint64_t above = mass([&](float z, int i) { return kept(z, i) && ordered_bits(z) > key; });
            const uint64_t each = w(value_of_ordered(key));
            // ranks of that value: kept while what is above them is below the limit
            const double ties = each ? ceil((limit - static_cast<double>(above)) / static_cast<double>(each)) : 1.0;
            const int want = ties < 1.0 ? 1 : (ties > static_cast<double>(V) ? V : static_cast<int>(ties));
            int id = 0;
            for (int bit = 30; bit >= 0; --bit) {
                const int c2 = id + (1 << bit);
                if (c2 < V &&
                    count([&](float z, int i) { return kept(z, i) && ordered_bits(z) == key && i < c2; }) < want)
                    id = c2;
            }
            kept.key = key, kept.id = id;
        }
        if (min_p > 0.f) {
            // w >= min_p as a least logit, rounded up to a float; the largest logit stays
            const double least = static_cast<double>(m) + static_cast<double>(tau) * log(static_cast<double>(min_p));
            kept.least = __double2float_ru(least);
            if (min_p >= 1.f) kept.least = m;
            if (min_p > 1.f) kept.key = static_cast<uint32_t>(best >> 32), kept.id = key_id(best);
        }
        const uint64_t total = mass(kept);
        // first id whose cumulative kept weight passes u * total
        const uint64_t target = static_cast<uint64_t>(static_cast<double>(u) * static_cast<double>(total));
        const int each = ((V + kSampleThreads - 1) / kSampleThreads);
        uint64_t s = 0;
        for (int k = 0; k < each; ++k) {
            const int i = tid * each + k;
            const float z = i < V ? load_logit<D>(P.logits, at + i) : -INFINITY;
            const bool in = i < V && z > -INFINITY && kept(z, i);
            const uint64_t x = w(in ? z : m);
            s += in ? x : 0;
        }
        scan[tid] = s;
        if (tid == 0) hit_thread = -1;
        __syncthreads();
        if (tid == 0) {
            uint64_t run = 0;
            for (int k = 0; k < kSampleThreads; ++k) {
                if (run + scan[k] > target) {
                    hit_thread = k, hit_before = run;
                    break;
                }
                run += scan[k];
            }
        }
        __syncthreads();
        if (hit_thread >= 0) {
            uint64_t run = hit_before;
            int found = -1;
            for (int k = 0; k < each; ++k) {
                const int i = hit_thread * each + k;
                const float z = i < V ? load_logit<D>(P.logits, at + i) : -INFINITY;
                const bool in = i < V && z > -INFINITY && kept(z, i);
                const uint64_t x = w(in ? z : m);
                run += in ? x : 0;
                if (found < 0 && run > target) found = i;
            }
            token = found;
        }
        if (tid == 0 && P.prob) {
            const double z = static_cast<double>(load_logit<D>(P.logits, at + token));
            prob = static_cast<float>(exp((z - static_cast<double>(m)) / static_cast<double>(tau)) *
                                      8796093022208.0 / static_cast<double>(total));
        }
    }
    if (tid == 0) {
        P.tokens[row] = token;
        if (P.prob) P.prob[row] = prob;
    }
    if (P.filtered)
        for (int i = tid; i < V; i += kSampleThreads) {
            const float z = load_logit<D>(P.logits, at + i);
            store_logit<D>(P.filtered, at + i, kept(z, i) && z > -INFINITY ? z : SSD_DROPPED_LOGIT);
        }
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
    const SampleParams P{logits,   rows,     V,      ld,   temperature, top_k,    top_p,
                         min_p,    uniforms, tokens, prob, filtered,    dev_status};
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (dtype == SSD_F32)
        sample_kernel<F32Tag><<<static_cast<unsigned>(rows), kSampleThreads, 0, s>>>(P);
    else
        sample_kernel<BF16Tag><<<static_cast<unsigned>(rows), kSampleThreads, 0, s>>>(P);
    return launched();
}
