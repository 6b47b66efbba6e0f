// ssd_kv_attend.cu -- attention of new tokens over the paged e4m3 cache (sm_103a).
//
//   s_j = sm_scale <q, k8_j> ks(page j),   out = sum_j softmax(s)_j v8_j vs(page j)
//
// One warp takes one token and query head and walks the positions 32 at a time: a lane
// scores one key, the warp keeps the running maximum and sum of the softmax, and each
// lane then gathers D / 32 channels of the values.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "ssd_kv.h"

namespace ssd {
namespace {

constexpr size_t kWorkspace = 256;
constexpr int kAttendThreads = 128;

struct AttendParams {
    const void *q;
    int64_t q_stride;
    const uint8_t *k, *v;
    const float *ks, *vs;
    int num_pages, page_shift, Hq, Hkv;
    const int32_t *table;
    int max_blocks;
    const int32_t *cu, *kv_len;
    int B, T, max_new;
    float scale;
    int window;
    void *out;
    int32_t *dev_status;
};

__device__ __forceinline__ float wide(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float wide(__half x) { return __half2float(x); }
__device__ __forceinline__ void narrow(float x, __nv_bfloat16 *p) { *p = __float2bfloat16(x); }
__device__ __forceinline__ void narrow(float x, __half *p) { *p = __float2half(x); }
__device__ __forceinline__ float e4m3_value(uint32_t byte) {
    const uint32_t h = halves_of_e4m3x2(byte);
    return __half2float(__ushort_as_half(static_cast<unsigned short>(h & 0xFFFFu)));
}

template <class E, int D>
__global__ void __launch_bounds__(kAttendThreads) attend_kernel(const __grid_constant__ AttendParams P) {
    __shared__ float qs[kAttendThreads / 32][D];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t id = static_cast<int64_t>(blockIdx.x) * (kAttendThreads / 32) + warp;
    if (id >= static_cast<int64_t>(P.T) * P.Hq) return;
    const int t = static_cast<int>(id / P.Hq), h = static_cast<int>(id % P.Hq);
    const int hk = h / (P.Hq / P.Hkv);
    // the sequence of token t: the last b with cu[b] <= t
    int lo = 0, hi = P.B;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (P.cu[mid] <= t)
            lo = mid;
        else
            hi = mid;
    }
    const int b = lo;
    const int first = P.cu[b], end = P.cu[b + 1];
    const int n = end - first, i = t - first;
    E *out = static_cast<E *>(P.out) + (static_cast<int64_t>(t) * P.Hq + h) * D;
    float acc[D / 32];
#pragma unroll
    for (int c = 0; c < D / 32; ++c) acc[c] = 0.f;
    float m = -INFINITY, l = 0.f;
    const bool real = t >= first && t < end && i < P.max_new;
    if (i == 0 && n > P.max_new && lane == 0) report(P.dev_status, SSD_DEV_BAD_LENGTH);
    if (real) {
        const int kv = min(P.kv_len[b], P.max_blocks << P.page_shift);
        const int pos = P.kv_len[b] - n + i;
        const int stop = min(pos + 1, kv);
        const int start = P.window > 0 ? max(0, pos + 1 - P.window) : 0;
        const E *q = static_cast<const E *>(P.q) + static_cast<int64_t>(t) * P.q_stride + static_cast<int64_t>(h) * D;
        for (int c = lane; c < D; c += 32) qs[warp][c] = wide(q[c]);
        __syncwarp();
        const int mask = (1 << P.page_shift) - 1;
        for (int j0 = start; j0 < stop; j0 += 32) {
            const int j = j0 + lane;
            float s = -INFINITY, vscale = 0.f;
            int64_t row = -1;
            if (j < stop) {
                const int page = P.table[static_cast<int64_t>(b) * P.max_blocks + (j >> P.page_shift)];
                if (page >= 0 && page < P.num_pages) {
                    const int64_t block = static_cast<int64_t>(page) * P.Hkv + hk;
                    row = (block << P.page_shift) + (j & mask);
                    const uint4 *k = reinterpret_cast<const uint4 *>(P.k + row * D);
                    float dot = 0.f;
                    for (int c = 0; c < D / 16; ++c) {
                        const uint4 w = __ldg(k + c);
                        const uint32_t r[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                        for (int e = 0; e < 16; ++e)
                            dot = fmaf(qs[warp][c * 16 + e], e4m3_value((r[e >> 2] >> (8 * (e & 3))) & 0xFFu), dot);
                    }
                    s = dot * P.ks[block] * P.scale;
                    vscale = P.vs[block];
                } else {
                    report(P.dev_status, SSD_DEV_BAD_PAGE);
                }
            }
            float top = s;
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
            const float m2 = fmaxf(m, top);
            if (m2 == -INFINITY && !__any_sync(0xFFFFFFFFu, s != s)) continue;
            const float ref = m2 == -INFINITY ? 0.f : m2;
            const float back = m == -INFINITY ? 0.f : expf(m - ref);
            float p = row >= 0 ? expf(s - ref) : 0.f;
            float sum = p;
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
            l = l * back + sum;
            m = m2;
#pragma unroll
            for (int c = 0; c < D / 32; ++c) acc[c] *= back;
            const float w = p * vscale;
            for (int k = 0; k < 32; ++k) {
                const float wk = __shfl_sync(0xFFFFFFFFu, w, k);
                const int64_t rk = __shfl_sync(0xFFFFFFFFu, row, k);
                if (rk < 0) continue;
#pragma unroll
                for (int c = 0; c < D / 32; ++c) acc[c] = fmaf(wk, e4m3_value(P.v[rk * D + c * 32 + lane]), acc[c]);
            }
        }
    }
    const float inv = l == 0.f ? 0.f : 1.f / l;
#pragma unroll
    for (int c = 0; c < D / 32; ++c) narrow(l == 0.f ? 0.f : acc[c] * inv, out + c * 32 + lane);
}

template <class E, int D>
int attend_launch(const AttendParams &P, cudaStream_t stream) {
    const int64_t warps = static_cast<int64_t>(P.T) * P.Hq;
    const int64_t blocks = (warps + 3) / 4;
    if (blocks > 0x7FFFFFFF) return SSD_ERR_UNSUPPORTED;
    attend_kernel<E, D><<<static_cast<unsigned>(blocks), kAttendThreads, 0, stream>>>(P);
    return launched();
}

}  // namespace
}  // namespace ssd

extern "C" size_t ssd_kv_workspace_size(void) { return ssd::kWorkspace; }

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
    if (!workspace || !aligned(workspace, 256) || workspace_bytes < kWorkspace) return SSD_ERR_WORKSPACE;
    if (static_cast<int64_t>(num_pages) * page_size > 0x7FFFFFFF ||
        static_cast<int64_t>(num_pages) * Hkv > 0x7FFFFFFF / page_size ||
        static_cast<int64_t>(B) * max_blocks > 0x7FFFFFFF || static_cast<int64_t>(max_blocks) * page_size > 0x7FFFFFFF ||
        B > SSD_KV_MAX_B)
        return SSD_ERR_UNSUPPORTED;
    if (T == 0) return SSD_OK;
    const AttendParams P{q,
                         q_stride,
                         static_cast<const uint8_t *>(k_cache),
                         static_cast<const uint8_t *>(v_cache),
                         k_scale,
                         v_scale,
                         num_pages,
                         log2_of(page_size),
                         Hq,
                         Hkv,
                         block_table,
                         max_blocks,
                         cu_new,
                         kv_len,
                         B,
                         T,
                         max_new,
                         sm_scale,
                         window,
                         out,
                         dev_status};
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (dtype == SSD_BF16)
        return D == 64 ? attend_launch<__nv_bfloat16, 64>(P, s) : attend_launch<__nv_bfloat16, 128>(P, s);
    return D == 64 ? attend_launch<__half, 64>(P, s) : attend_launch<__half, 128>(P, s);
}
