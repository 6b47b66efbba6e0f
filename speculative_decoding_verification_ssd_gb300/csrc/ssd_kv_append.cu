// ssd_kv_append.cu -- new keys and values into the paged e4m3 cache (sm_103a).
//
// One scale stands for a whole (page, head) block, so a block's new tokens are looked at
// together: their largest magnitude gives the smallest power of two that brings them into
// e4m3's range, and where that exceeds the block's scale the tokens already there are
// stored again under the new one.  A power of two costs e4m3 no precision (the format
// floats), and makes that second rounding exact but for the smallest values.
//
// A warp takes one run (the tokens of one page, found from the slots alone: a run starts
// where the page differs from the token before), one head, and keys or values.  Its lanes
// hold 8 channels each, 16 bytes in and 8 bytes out, 256 / D tokens at a time; kHold of
// those steps are under way together, and stay in registers between the search for the
// largest magnitude and the conversion where the run has no more.
//
// What bounds it is the chain of dependent reads (slots, then the old scale and the tokens
// together), a decoded token's (8 us captured into a graph with L2 flushed, 7 of it an empty
// launch) and, four waves of warps after one another, a prompt's: 12 of 1365 tokens, 8 heads
// of 128 in pages of 32, take 26 us, 3.9 TB/s (fp32 43, 3.9).  Hence one look at 32 slots by the lanes names
// a run's start, page and, as a rule, end.  Measured, for that prompt: the end looked for
// in a second read, before any token's, 32 us; 8 steps under way 54, 16 33; CTAs of 2, 4, 8
// and 16 warps 35, 32, 33 and 35; CTAs that stay and take chunk after chunk 27 (54, against
// 35, in pages of 128, where few chunks start a run).
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "ssd_kv.h"

namespace ssd {
namespace {

constexpr int kAppendThreads = 128;
constexpr int kAppendCtas = 4;  // to an SM, which leaves a thread the registers of its steps
constexpr int kHold = 16;       // steps under way together, whose values stay in registers

struct AppendParams {
    const void *x[2];  // keys, values
    int64_t stride[2];
    const int32_t *slots;
    int T, H;
    uint8_t *cache[2];
    float *scale[2];
    int num_pages;
    int page_shift;
    int chunk_shift;  // tokens that one warp looks through for starts of runs: 1 << chunk_shift
    int64_t units;    // chunks * H * 2
    int32_t *dev_status;
};


__device__ __forceinline__ float wide(float x) { return x; }
__device__ __forceinline__ float wide(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float wide(__half x) { return __half2float(x); }

// Eight values as they lie in memory.
template <class E>
struct Raw {
    static constexpr int kWords = static_cast<int>(sizeof(E)) * 2;
    uint32_t w[kWords];
};
template <class E, bool kVec>
__device__ __forceinline__ void load8(const E *p, Raw<E> &r) {
    if (kVec) {
#pragma unroll
        for (int i = 0; i < Raw<E>::kWords; i += 4) {
            const uint4 a = __ldcs(reinterpret_cast<const uint4 *>(p) + i / 4);
            r.w[i] = a.x, r.w[i + 1] = a.y, r.w[i + 2] = a.z, r.w[i + 3] = a.w;
        }
    } else {
        E *v = reinterpret_cast<E *>(r.w);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = p[i];
    }
}
template <class E>
__device__ __forceinline__ void widen(const Raw<E> &r, float (&v)[8]) {
    const E *e = reinterpret_cast<const E *>(r.w);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = wide(e[i]);
}

// Largest finite magnitude; `odd` is set when a value is not finite.
__device__ __forceinline__ void magnitude(const float (&v)[8], float &amax, bool &odd) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float a = fabsf(v[i]);
        const bool fine = a <= 3.402823466e38f;
        odd |= !fine;
        if (fine) amax = fmaxf(amax, a);
    }
}

// The same of values as they lie in memory.  Without their signs, halves of either kind order as whole numbers, so
// two are compared at once; what reaches the pattern of infinity is looked at again, value by value.
template <class E>
__device__ __forceinline__ uint32_t infinity_bits();
template <>
__device__ __forceinline__ uint32_t infinity_bits<__nv_bfloat16>() {
    return 0x7F80u;
}
template <>
__device__ __forceinline__ uint32_t infinity_bits<__half>() {
    return 0x7C00u;
}
template <class E, int kN>
__device__ __forceinline__ void magnitudes(const Raw<E> (&r)[kN], float &amax, bool &odd) {
    if constexpr (sizeof(E) == 2) {
        uint32_t top = 0;
#pragma unroll
        for (int i = 0; i < kN; ++i)
#pragma unroll
            for (int c = 0; c < Raw<E>::kWords; ++c) top = __vmaxu2(top, r[i].w[c] & 0x7FFF7FFFu);
        const uint32_t most = max(top & 0xFFFFu, top >> 16);
        if (most < infinity_bits<E>()) {
            const uint16_t bits = static_cast<uint16_t>(most);
            amax = fmaxf(amax, wide(*reinterpret_cast<const E *>(&bits)));
            return;
        }
    }
#pragma unroll
    for (int i = 0; i < kN; ++i) {
        float v[8];
        widen(r[i], v);
        magnitude(v, amax, odd);
    }
}

// The smallest power of two 2^k, k >= -100, with amax <= 448 * 2^k.  448 is 1.75 * 2^8: the
// exponent decides, and the mantissa whether it has to be the next one.
__device__ __forceinline__ float needed_scale(float amax) {
    const uint32_t u = __float_as_uint(amax);
    int k = static_cast<int>(u >> 23) - 127 - 8 + ((u & 0x7FFFFFu) > 0x600000u ? 1 : 0);
    k = k < -100 ? -100 : k;
    return __uint_as_float(static_cast<uint32_t>(k + 127) << 23);
}

__device__ __forceinline__ uint2 pack8(const float (&v)[8], float inv) {
    uint2 r;
    r.x = e4m3x2(v[0] * inv, v[1] * inv) | (e4m3x2(v[2] * inv, v[3] * inv) << 16);
    r.y = e4m3x2(v[4] * inv, v[5] * inv) | (e4m3x2(v[6] * inv, v[7] * inv) << 16);
    return r;
}
// A scale that the cache held before need not be a power of two: divide.
__device__ __forceinline__ uint2 pack8_div(const float (&v)[8], float scale) {
    float q[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) q[i] = __fdiv_rn(v[i], scale);
    return pack8(q, 1.f);
}

template <class E, int D, bool kVec>
__global__ void __launch_bounds__(kAppendThreads, kAppendCtas) append_kernel(const __grid_constant__ AppendParams P) {
    constexpr int kLanes = D / 8;          // lanes of one token
    constexpr int kStep = 32 / kLanes;     // tokens of one step
    const int lane = threadIdx.x & 31;
    const int sub = lane / kLanes, ch = (lane % kLanes) * 8;
    const int chunk = 1 << P.chunk_shift;
    const int64_t cache_rows = static_cast<int64_t>(P.num_pages) << P.page_shift;
    const int page_mask = (1 << P.page_shift) - 1;

    const int64_t unit = (static_cast<int64_t>(blockIdx.x) * kAppendThreads + threadIdx.x) >> 5;
    if (unit >= P.units) return;
    const int what = static_cast<int>(unit & 1);
    const int64_t rest = unit >> 1, at = rest / P.H;
    const int h = static_cast<int>(rest - at * P.H);
    const int64_t t0 = at << P.chunk_shift;
    const E *x = static_cast<const E *>(P.x[what]);
    const int64_t stride = P.stride[what];

    // the chunk's tokens and those after it, one per lane: the page of each, -1 for a slot that is skipped
    auto page_of = [&](int slot) { return slot >= 0 && slot < cache_rows ? slot >> P.page_shift : -1; };
    const int slot = t0 + lane < P.T ? P.slots[t0 + lane] : -1;
    int before = lane == 0 && t0 > 0 ? P.slots[t0 - 1] : -1;
    if (slot >= cache_rows) report(P.dev_status, SSD_DEV_BAD_PAGE);
    const int page = page_of(slot), up = __shfl_up_sync(0xFFFFFFFFu, slot, 1);
    if (lane > 0) before = up;
    uint32_t starts = __ballot_sync(0xFFFFFFFFu, lane < chunk && page >= 0 && page != page_of(before));
    while (starts) {
        const int leader = __ffs(starts) - 1;
        starts &= starts - 1;
        const int64_t t = t0 + leader;
        const int p = __shfl_sync(0xFFFFFFFFu, page, leader);
        const int row0 = __shfl_sync(0xFFFFFFFFu, slot, leader) & page_mask;
        const int64_t block = static_cast<int64_t>(p) * P.H + h;
        float *scale_at = P.scale[what] + block;
        const float scale_was = *scale_at;
        uint8_t *rows = P.cache[what] + ((block << P.page_shift) * D);
        const E *xt = x + t * stride + static_cast<int64_t>(h) * D + ch;

        // kSteps steps of tokens from k0 on; those beyond the run are zero
        constexpr int kSteps = sizeof(E) == 4 ? kHold / 2 : kHold;
        Raw<E> hold[kSteps];
        auto fetch = [&](int k0, int end) {
#pragma unroll
            for (int i = 0; i < kSteps; ++i) {
                const int k = k0 + i * kStep + sub;
                if (k < end) {
                    load8<E, kVec>(xt + k * stride, hold[i]);
                } else {
#pragma unroll
                    for (int c = 0; c < Raw<E>::kWords; ++c) hold[i].w[c] = 0u;
                }
            }
        };
        // Length of the run: tokens from t on with the same page.  Where it passes what the lanes see, the first steps
        // go up to the page's last row, which ends a run whose slots ascend, and are on their way while the rest is
        // looked up.
        const uint32_t differ = ~(__ballot_sync(0xFFFFFFFFu, page == p) >> leader);
        const int seen = 32 - leader;
        int n = differ ? __ffs(differ) - 1 : 32;
        int end = n;
        if (n == seen) end = max(seen, static_cast<int>(min(static_cast<int64_t>(page_mask + 1 - row0), P.T - t)));
        fetch(0, end);
        if (n == seen) {
            for (;;) {
                const int64_t tt = t + n + lane;
                const uint32_t m = __ballot_sync(0xFFFFFFFFu, tt < P.T && page_of(P.slots[tt]) == p);
                if (m != 0xFFFFFFFFu) {
                    n += __ffs(~m) - 1;
                    break;
                }
                n += 32;
            }
            if (n != end && min(n, end) < kSteps * kStep) fetch(0, n);
        }
        float amax = 0.f;
        bool odd = false;
        for (int k0 = 0; k0 < n; k0 += kSteps * kStep) {
            if (k0 > 0) fetch(k0, n);
            magnitudes(hold, amax, odd);
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, o));
        if (__any_sync(0xFFFFFFFFu, odd) && lane == 0) report(P.dev_status, SSD_DEV_NONFINITE);

        const float need = needed_scale(amax);
        const bool had = row0 > 0 && scale_was > 0.f && scale_was <= 3.402823466e38f;
        const float scale = had && scale_was > need ? scale_was : need;
        if (row0 > 0 && !(had && scale_was == scale)) {
            const float ratio = had ? __fdiv_rn(scale_was, scale) : 0.f;
            for (int r = sub; r < row0; r += kStep) {
                uint2 *at = reinterpret_cast<uint2 *>(rows + static_cast<int64_t>(r) * D + ch);
                const uint2 w = *at;
                float v[8];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const uint32_t two = halves_of_e4m3x2(((i < 2 ? w.x : w.y) >> (16 * (i & 1))) & 0xFFFFu);
                    const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&two));
                    v[2 * i] = f.x, v[2 * i + 1] = f.y;
                }
                *at = pack8(v, ratio);
            }
        }
        const bool pow2 = (__float_as_uint(scale) & 0x7FFFFFu) == 0 && scale >= 7.8e-31f;
        const float inv = pow2 ? __frcp_rn(scale) : 0.f;
        auto store = [&](int k, const float(&v)[8]) {
            const int s = __ldg(P.slots + t + k);
            uint2 *at = reinterpret_cast<uint2 *>(rows + static_cast<int64_t>(s & page_mask) * D + ch);
            *at = pow2 ? pack8(v, inv) : pack8_div(v, scale);
        };
        for (int k0 = 0; k0 < n; k0 += kSteps * kStep) {
            if (n > kSteps * kStep) fetch(k0, n);  // else they are still there
#pragma unroll
            for (int i = 0; i < kSteps; ++i) {
                const int k = k0 + i * kStep + sub;
                float v[8];
                widen(hold[i], v);
                if (k < n) store(k, v);
            }
        }
        if (lane == 0 && !(scale_was == scale)) *scale_at = scale;
    }
}

template <class E, int D>
int append_launch(const AppendParams &P, bool vec, cudaStream_t stream) {
    const int64_t blocks = (P.units * 32 + kAppendThreads - 1) / kAppendThreads;
    if (blocks > 0x7FFFFFFF) return SSD_ERR_UNSUPPORTED;
    if (vec)
        append_kernel<E, D, true><<<static_cast<unsigned>(blocks), kAppendThreads, 0, stream>>>(P);
    else
        append_kernel<E, D, false><<<static_cast<unsigned>(blocks), kAppendThreads, 0, stream>>>(P);
    return launched();
}

}  // namespace
}  // namespace ssd

extern "C" int ssd_kv_append(const void *k, const void *v, int dtype, int64_t k_stride, int64_t v_stride,
                             const int32_t *slots, int T, int Hkv, int D, void *k_cache, void *v_cache, float *k_scale,
                             float *v_scale, int num_pages, int page_size, int32_t *dev_status, void *stream) {
    using namespace ssd;
    if (dtype != SSD_F32 && dtype != SSD_BF16 && dtype != SSD_F16) return SSD_ERR_DTYPE;
    if (T < 0 || Hkv < 1 || num_pages < 1 || !kv_page_size_ok(page_size) || (D != 64 && D != 128))
        return SSD_ERR_INVALID_ARG;
    if (!k_cache || !v_cache || !k_scale || !v_scale || (T > 0 && (!k || !v || !slots))) return SSD_ERR_INVALID_ARG;
    if (!aligned(k_cache, 16) || !aligned(v_cache, 16)) return SSD_ERR_INVALID_ARG;
    if (T > 1 && (k_stride < static_cast<int64_t>(Hkv) * D || v_stride < static_cast<int64_t>(Hkv) * D))
        return SSD_ERR_INVALID_ARG;
    if (static_cast<int64_t>(num_pages) * page_size > 0x7FFFFFFF ||
        static_cast<int64_t>(num_pages) * Hkv > 0x7FFFFFFF / page_size)
        return SSD_ERR_UNSUPPORTED;
    if (T == 0) return SSD_OK;
    AppendParams P{};
    P.x[0] = k, P.x[1] = v;
    P.stride[0] = k_stride, P.stride[1] = v_stride;
    P.slots = slots;
    P.T = T, P.H = Hkv;
    P.cache[0] = static_cast<uint8_t *>(k_cache), P.cache[1] = static_cast<uint8_t *>(v_cache);
    P.scale[0] = k_scale, P.scale[1] = v_scale;
    P.num_pages = num_pages;
    P.page_shift = log2_of(page_size);
    // As many tokens per warp as still leave 64 warps to each of 152 SMs, four times what is resident: a decoded token is
    // a run of its own, and runs met by one warp follow one another.  Leaving 16, 32, 64 and 128 warps, 256 x 5 tokens
    // take 14.9, 13.1, 14.9 and 16.9 us, one prompt of 1365 tokens 11.1, 12.8, 13.3 and 17.2, 12 of them 27.1, 27.1,
    // 27.1 and 31.4.
    P.chunk_shift = 0;
    while (P.chunk_shift < 4 && ((static_cast<int64_t>(T) * Hkv * 2) >> (P.chunk_shift + 1)) >= 64 * 152) ++P.chunk_shift;
    P.units = ((static_cast<int64_t>(T) + (1 << P.chunk_shift) - 1) >> P.chunk_shift) * Hkv * 2;
    P.dev_status = dev_status;
    const int es = dtype == SSD_F32 ? 4 : 2;
    const bool vec = aligned(k, 16) && aligned(v, 16) && k_stride * es % 16 == 0 && v_stride * es % 16 == 0;
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (dtype == SSD_F32) return D == 64 ? append_launch<float, 64>(P, vec, s) : append_launch<float, 128>(P, vec, s);
    if (dtype == SSD_BF16)
        return D == 64 ? append_launch<__nv_bfloat16, 64>(P, vec, s) : append_launch<__nv_bfloat16, 128>(P, vec, s);
    return D == 64 ? append_launch<__half, 64>(P, vec, s) : append_launch<__half, 128>(P, vec, s);
}
