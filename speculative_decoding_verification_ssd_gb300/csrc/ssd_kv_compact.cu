// ssd_kv_compact.cu -- an accepted path's keys and values to the rows after the committed ones of
// the paged e4m3 cache (sm_103a).
//
// A warp takes one sequence, one head, and keys or values.  It reads the whole path into registers
// before it writes a row, since a row may be the source of one node and the place of another; its
// pages are its alone.  Tokens that stay in their page keep their bytes; those that come from
// another bring its scale along, and where that asks for a larger one the page's earlier rows are
// stored again under it, as the append does.
//
// Bound by latency: the accepted length, the path, the table, the sources' scales and rows, and the
// destination's scale are read one after another, each a miss when the caches are cold (the path need
// not wait for the length, nor the last scale for the rows).  256 sequences of 8 heads of 128, paths of up to 9, move 4.7 MB at
// most (0.7 us at the copy's rate): 11.4 us with cold caches, of which an almost empty kernel makes 7,
// and one sequence of 4 heads 9.3.  The steps of 4 or 8 tokens end with the path: a form that went
// over all SSD_MAX_K took 15.5 us.  72 or 64 registers, with which every warp is resident at once, and
// four steps of a restored page on their way change nothing.
#include <cuda_fp16.h>

#include "ssd_kv.h"

namespace ssd {
namespace {

constexpr int kCompactThreads = 128;
constexpr float kMost = 3.402823466e38f;

struct CompactParams {
    const int32_t *path, *accept_len, *seq_len, *table;
    int B, max_path, max_blocks, H;
    uint8_t *cache[2];
    float *scale[2];
    int num_pages, page_shift;
    int64_t units;  // B * H * 2
    int32_t *dev_status;
};

// A byte times a large scale may pass fp32 (a bf16 value next to its type's largest is held so): magnitudes are 2^-kDown of
// theirs.  What that makes inexact is far below the smallest need.
constexpr int kDown = 16;
constexpr float kDownBy = 1.f / (1 << kDown);

// The smallest power of two 2^k, -100 <= k <= 127, with amax <= 448 * 2^k (448 is 1.75 * 2^8), of 2^-kDown amax.
__device__ __forceinline__ float needed_scale(float amax) {
    const uint32_t u = __float_as_uint(amax);
    int k = static_cast<int>(u >> 23) + kDown - 127 - 8 + ((u & 0x7FFFFFu) > 0x600000u ? 1 : 0);
    k = min(max(k, -100), 127);
    return __uint_as_float(static_cast<uint32_t>(k + 127) << 23);
}

// Four e4m3 bytes as e4m3(x * by / over); over = 0: no quotient.
__device__ __forceinline__ uint32_t restored(uint32_t w, float by, float over) {
    float v[4];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const uint32_t two = halves_of_e4m3x2((w >> (16 * i)) & 0xFFFFu);
        const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&two));
        v[2 * i] = f.x * by, v[2 * i + 1] = f.y * by;
    }
    if (over != 0.f) {
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = __fdiv_rn(v[i], over);
    }
    return e4m3x2(v[0], v[1]) | (e4m3x2(v[2], v[3]) << 16);
}
__device__ __forceinline__ uint4 restored(uint4 w, float by, float over) {
    return make_uint4(restored(w.x, by, over), restored(w.y, by, over), restored(w.z, by, over), restored(w.w, by, over));
}

// Largest magnitude of four bytes, NaN left out, as the bits of a byte.
__device__ __forceinline__ uint32_t largest(uint32_t w) {
    w &= 0x7F7F7F7Fu;
    const uint32_t nan = (w + 0x01010101u) & 0x80808080u;
    return w & ~((nan >> 7) * 0xFFu);
}

template <int D>
__global__ void __launch_bounds__(kCompactThreads) compact_kernel(const __grid_constant__ CompactParams P) {
    constexpr uint32_t kAll = 0xFFFFFFFFu;
    constexpr int kLanes = D / 16;               // of one token, 16 bytes each
    constexpr int kStep = 32 / kLanes;           // tokens at a time
    constexpr int kSteps = SSD_MAX_K / kStep;
    const int lane = threadIdx.x & 31, sub = lane / kLanes, part = lane % kLanes;
    const int64_t unit = (static_cast<int64_t>(blockIdx.x) * kCompactThreads + threadIdx.x) >> 5;
    if (unit >= P.units) return;
    const int b = static_cast<int>(unit / (2 * P.H)), rest = static_cast<int>(unit - static_cast<int64_t>(b) * (2 * P.H));
    const int h = rest >> 1, what = rest & 1;
    const int page_rows = 1 << P.page_shift, page_mask = page_rows - 1;

    const int a = P.accept_len[b], keep = P.seq_len[b];
    const int32_t *path = P.path + static_cast<int64_t>(b) * P.max_path;
    if (a < 0) return;
    // node j + 1 of the path is this lane's; node 0 lies in place
    const int j = lane + 1;
    const int node = j <= a && j < P.max_path ? path[j] : -1;
    int before = __shfl_up_sync(kAll, node, 1);
    if (lane == 0) before = path[0];
    int bad = 0;
    if (a >= P.max_path || keep < 0) bad = SSD_DEV_BAD_LENGTH;
    const bool mine = bad == 0 && j <= a;
    if (mine && node <= before) bad |= SSD_DEV_BAD_TREE;
    if (lane == 0 && before != 0) bad |= SSD_DEV_BAD_TREE;
    const int64_t rows = static_cast<int64_t>(P.max_blocks) << P.page_shift;
    const int64_t from = static_cast<int64_t>(keep) + (mine ? node : 0), to = static_cast<int64_t>(keep) + (mine ? j : 0);
    if (!bad && (from >= rows || to >= rows)) bad = SSD_DEV_BAD_LENGTH;
    int from_page = 0, to_page = 0, first_page = 0;
    if (__any_sync(kAll, bad) == 0) {
        const int32_t *table = P.table + static_cast<int64_t>(b) * P.max_blocks;
        from_page = table[from >> P.page_shift], to_page = table[to >> P.page_shift];
        first_page = table[keep >> P.page_shift];
        if (from_page < 0 || from_page >= P.num_pages || to_page < 0 || to_page >= P.num_pages || first_page < 0 ||
            first_page >= P.num_pages)
            bad = SSD_DEV_BAD_PAGE;
    }
    if (__any_sync(kAll, bad)) {
        report(P.dev_status, bad);
        return;
    }
    if (a == 0) return;
    float *scale = P.scale[what];
    uint8_t *cache = P.cache[what];
    auto block = [&](int page) { return static_cast<int64_t>(page) * P.H + h; };
    const float from_scale = mine ? scale[block(from_page)] : 0.f;
    const int64_t from_row = (block(from_page) << P.page_shift) + (from & page_mask);
    const int64_t to_row = (block(to_page) << P.page_shift) + (to & page_mask);

    uint4 held[kSteps];
#pragma unroll
    for (int i = 0; i < kSteps; ++i) {
        if (i * kStep >= a) break;  // (the same for the warp)
        const int k = i * kStep + sub;  // lane that knows the token
        const int64_t row = __shfl_sync(kAll, from_row, k);
        held[i] = k < a ? *reinterpret_cast<const uint4 *>(cache + row * D + part * 16) : make_uint4(0, 0, 0, 0);
    }
    // largest magnitude of each token, at the lane that knows it
    float amax = 0.f;
    const bool comes = mine && from_page != to_page;
#pragma unroll
    for (int i = 0; i < kSteps; ++i) {
        if (i * kStep >= a) break;  // (the same for the warp)
        uint32_t m = __vmaxu4(__vmaxu4(largest(held[i].x), largest(held[i].y)), __vmaxu4(largest(held[i].z), largest(held[i].w)));
#pragma unroll
        for (int o = 1; o < kLanes; o <<= 1) m = __vmaxu4(m, __shfl_xor_sync(kAll, m, o));
        m = __vmaxu4(m, m >> 16);
        m = __vmaxu4(m, m >> 8) & 0xFFu;
        const uint32_t got = __shfl_sync(kAll, m, (lane % kStep) * kLanes);
        if (lane / kStep == i) {
            const uint32_t two = halves_of_e4m3x2(got);
            amax = __half22float2(*reinterpret_cast<const __half2 *>(&two)).x * (fabsf(from_scale) * kDownBy);
        }
    }
    if (!comes || !(amax <= kMost)) amax = 0.f;

    // the pages of the path's places, one after another: at most (SSD_MAX_K + 15) / 16 + 1
    const int q0 = keep >> P.page_shift, q1 = static_cast<int>((static_cast<int64_t>(keep) + a) >> P.page_shift);
    float ratio = 1.f, grown = from_scale;  // of the page that this lane's token goes to
    for (int q = q0; q <= q1; ++q) {
        const bool here = mine && static_cast<int>(to >> P.page_shift) == q;
        if (!__any_sync(kAll, here && comes)) continue;
        const uint32_t top = __reduce_max_sync(kAll, here ? __float_as_uint(amax) : 0u);
        const int page = q == q0 ? first_page : __shfl_sync(kAll, to_page, __ffs(__ballot_sync(kAll, here)) - 1);
        const float was = scale[block(page)], need = needed_scale(__uint_as_float(top));
        const bool had = was > 0.f && was <= kMost;
        const float now = had && was > need ? was : need;
        const float r = now == was ? 1.f : (had ? __fdiv_rn(was, now) : 0.f);
        if (here) ratio = r, grown = now;
        if (!(now == was)) {
            if (q == q0) {
                uint8_t *at = cache + (block(page) << P.page_shift) * D;
                for (int i = sub; i <= (keep & page_mask); i += kStep) {
                    uint4 *row = reinterpret_cast<uint4 *>(at + static_cast<int64_t>(i) * D + part * 16);
                    *row = restored(*row, r, 0.f);
                }
            }
            __syncwarp();
            if (lane == 0) scale[block(page)] = now;
        }
    }
    __syncwarp();
#pragma unroll
    for (int i = 0; i < kSteps; ++i) {
        if (i * kStep >= a) break;  // (the same for the warp)
        const int k = i * kStep + sub;
        const int64_t row = __shfl_sync(kAll, to_row, k), was = __shfl_sync(kAll, from_row, k);
        const bool other = __shfl_sync(kAll, comes, k);
        const float r = __shfl_sync(kAll, ratio, k), s = __shfl_sync(kAll, from_scale, k), over = __shfl_sync(kAll, grown, k);
        if (k >= a) continue;
        uint4 *to_at = reinterpret_cast<uint4 *>(cache + row * D + part * 16);
        if (other)
            // (the quotient of both's 2^-kDown is the same)
            *to_at = s == over ? held[i] : (s > 1.f ? restored(held[i], s * kDownBy, over * kDownBy) : restored(held[i], s, over));
        else if (r != 1.f)
            *to_at = restored(held[i], r, 0.f);
        else if (row != was)
            *to_at = held[i];
    }
}

}  // namespace
}  // namespace ssd

extern "C" int ssd_kv_compact(const int32_t *path, const int32_t *accept_len, const int32_t *seq_len, int B, int max_path,
                              const int32_t *block_table, int max_blocks, int Hkv, int D, void *k_cache, void *v_cache,
                              float *k_scale, float *v_scale, int num_pages, int page_size, int32_t *dev_status,
                              void *stream) {
    using namespace ssd;
    if (!path || !accept_len || !seq_len || !block_table || !k_cache || !v_cache || !k_scale || !v_scale) return SSD_ERR_INVALID_ARG;
    if (B < 1 || max_path < 1 || max_path > SSD_MAX_K + 1 || max_blocks < 1 || num_pages < 1 || Hkv < 1 ||
        !kv_page_size_ok(page_size) || (D != 64 && D != 128))
        return SSD_ERR_INVALID_ARG;
    if (!aligned(k_cache, 16) || !aligned(v_cache, 16)) return SSD_ERR_INVALID_ARG;
    if (B > SSD_KV_MAX_B || static_cast<int64_t>(num_pages) * page_size > 0x7FFFFFFF ||
        static_cast<int64_t>(num_pages) * Hkv > 0x7FFFFFFF / page_size || static_cast<int64_t>(B) * max_blocks > 0x7FFFFFFF ||
        static_cast<int64_t>(max_blocks) * page_size > 0x7FFFFFFF / 2)
        return SSD_ERR_UNSUPPORTED;
    CompactParams P{};
    P.path = path, P.accept_len = accept_len, P.seq_len = seq_len, P.table = block_table;
    P.B = B, P.max_path = max_path, P.max_blocks = max_blocks, P.H = Hkv;
    P.cache[0] = static_cast<uint8_t *>(k_cache), P.cache[1] = static_cast<uint8_t *>(v_cache);
    P.scale[0] = k_scale, P.scale[1] = v_scale;
    P.num_pages = num_pages, P.page_shift = log2_of(page_size);
    P.units = static_cast<int64_t>(B) * Hkv * 2;
    P.dev_status = dev_status;
    const int64_t blocks = (P.units * 32 + kCompactThreads - 1) / kCompactThreads;
    if (blocks > 0x7FFFFFFF) return SSD_ERR_UNSUPPORTED;
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (D == 64)
        compact_kernel<64><<<static_cast<unsigned>(blocks), kCompactThreads, 0, s>>>(P);
    else
        compact_kernel<128><<<static_cast<unsigned>(blocks), kCompactThreads, 0, s>>>(P);
    return launched();
}
