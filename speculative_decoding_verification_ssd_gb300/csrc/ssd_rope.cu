// ssd_rope.cu -- norm of each query and key head and its rotation by the token's position
// (sm_103a).
//
//   y = x rsqrt(mean x^2 + eps) w,   (a, b) -> (a cos t - b sin t, a sin t + b cos t),  t = 2 pi pos f_i
//
// A frequency f_i is held in turns, as a 64-bit fraction: pos * f_i in 64-bit integers drops the
// whole turns exactly, and what is left has 32 bits however far the position is (an fp32 angle at
// position 10^5 is off by 2^-8; its reduction in fp64 costs 64 times the fp32 rate here).
//
// A lane holds 16 channels of a head in two runs of 8: of halves the runs that are turned with each
// other, of neighbours runs that hold their own pairs, so that no value crosses lanes but the sum of
// squares.  Sums and the rotation are fp32, two to an instruction, rounded once at the store; a head
// whose squares fp32 does not hold is done over at the end.
//
// A warp takes a token, D/16 lanes a head, and goes over the heads with the next pass's on their way:
// the angles (8 sincospi per lane) serve all of a token's heads.  Only while tokens alone would leave
// SMs idle does a warp take a slice of them and angles are made more than once (the rule is at its
// place).  Weights lie in shared memory: read per pass from global memory, 4 bytes to a lane, they
// were most of its loads (44 us, 40 with them here and 48 with both heads' held in registers).
//
// Bound by bytes: 9472 tokens of 32 + 8 heads of 128 in bf16 read and write 194 MB, 29 us at the
// copy's rate; 39 us, 5.0 TB/s, with the launch and a last wave that is not full (3648 warps are
// resident).  In fp32, half as many tokens, 34 to 38 us.  Tried: runs of 4 channels, half the
// registers (46 us); two and four passes on their way (42 and 69); 1, 5 and 8 blocks per SM asked
// for (40, 40, 44).  One token 7 to 9 us, a launch's own time.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "ssd_kv.h"

namespace ssd {
namespace {

constexpr int kRopeThreads = 128;
constexpr int kRopeBlocks = 6;  // per SM: 80 registers

struct RopeParams {
    const void *x[2];  // queries, keys
    void *y[2];
    int64_t x_stride[2], y_stride[2];
    const float *w[2];
    const int32_t *positions;
    const uint64_t *turns;
    int T, Hq, H;     // H: heads of both
    int R;            // pairs turned
    int interleaved;  // pairs are neighbours (else a half apart)
    float eps;
    int slices;       // warps that share a token
    int64_t units;    // T * slices
};

__device__ __forceinline__ float wide(float x) { return x; }
__device__ __forceinline__ float wide(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float wide(__half x) { return __half2float(x); }
__device__ __forceinline__ void narrow(float2 x, float *y) { y[0] = x.x, y[1] = x.y; }
__device__ __forceinline__ void narrow(float2 x, __nv_bfloat16 *y) { *reinterpret_cast<__nv_bfloat162 *>(y) = __float22bfloat162_rn(x); }
__device__ __forceinline__ void narrow(float2 x, __half *y) { *reinterpret_cast<__half2 *>(y) = __float22half2_rn(x); }

// Two fp32 products, or sums of products, of one instruction, each rounded as fmaf rounds.
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
    uint64_t d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;"
        : "=l"(d)
        : "l"(reinterpret_cast<uint64_t &>(a)), "l"(reinterpret_cast<uint64_t &>(b)), "l"(reinterpret_cast<uint64_t &>(c)));
    return reinterpret_cast<float2 &>(d);
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
    uint64_t d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(reinterpret_cast<uint64_t &>(a)), "l"(reinterpret_cast<uint64_t &>(b)));
    return reinterpret_cast<float2 &>(d);
}

// Eight values as they lie in memory.
template <class E>
struct Raw {
    alignas(16) E e[8];
};
template <class E, bool kVec>
__device__ __forceinline__ void load8(const E *p, Raw<E> &v) {
    if (kVec) {
#pragma unroll
        for (int i = 0; i < static_cast<int>(sizeof(E)) / 2; ++i)
            reinterpret_cast<uint4 *>(v.e)[i] = __ldcs(reinterpret_cast<const uint4 *>(p) + i);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) v.e[i] = p[i];
    }
}
template <class E, bool kVec>
__device__ __forceinline__ void store8(E *p, const float2 (&v)[4]) {
    alignas(16) E e[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) narrow(v[i], e + 2 * i);
    if (kVec) {
#pragma unroll
        for (int i = 0; i < static_cast<int>(sizeof(E)) / 2; ++i)
            reinterpret_cast<uint4 *>(p)[i] = reinterpret_cast<const uint4 *>(e)[i];
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) p[i] = e[i];
    }
}

// Cosines and sines of a lane's pairs, and the sines' negatives.
struct Turns {
    float2 c[4], s[4], n[4];
};
__device__ __forceinline__ Turns turns_of(const RopeParams &P, int t, int u) {
    Turns r;
    const uint64_t pos = static_cast<uint64_t>(static_cast<int64_t>(P.positions[t]));
    auto one = [&](int i, float &sine, float &cosine) {
        const int f = P.interleaved ? (i < 4 ? 4 * u + i : P.R / 2 + 4 * u + i - 4) : 8 * u + i;
        const int32_t left = static_cast<int32_t>((pos * __ldg(P.turns + f)) >> 32);
        sincospif(static_cast<float>(left) * 4.656612873077393e-10f, &sine, &cosine);  // 2^-31: half turns
    };
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        one(2 * i, r.s[i].x, r.c[i].x), one(2 * i + 1, r.s[i].y, r.c[i].y);
        r.n[i] = make_float2(-r.s[i].x, -r.s[i].y);
    }
    return r;
}
__device__ __forceinline__ void turn(const RopeParams &P, const Turns &t, float2 (&v)[4], float2 (&z)[4]) {
    if (P.interleaved) {
        auto rotate = [](float2 &p, float cosine, float sine) {
            p = make_float2(p.x * cosine - p.y * sine, p.x * sine + p.y * cosine);
        };
        rotate(v[0], t.c[0].x, t.s[0].x), rotate(v[1], t.c[0].y, t.s[0].y), rotate(v[2], t.c[1].x, t.s[1].x), rotate(v[3], t.c[1].y, t.s[1].y);
        rotate(z[0], t.c[2].x, t.s[2].x), rotate(z[1], t.c[2].y, t.s[2].y), rotate(z[2], t.c[3].x, t.s[3].x), rotate(z[3], t.c[3].y, t.s[3].y);
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 v0 = v[i], z0 = z[i];
            v[i] = fma2(v0, t.c[i], mul2(z0, t.n[i]));
            z[i] = fma2(v0, t.s[i], mul2(z0, t.c[i]));
        }
    }
}

// The lane's two runs of channels, and whether they are turned.
struct Runs {
    bool turned;
    int a, b;
};
template <int D>
__device__ __forceinline__ Runs runs_of(const RopeParams &P, int u) {
    const bool turned = u < P.R / 8;
    return {turned, turned ? 8 * u : P.R + 8 * u, turned ? P.R + 8 * u : D / 2 + 8 * u};
}
// A lane's head in a pass.
template <int D>
__device__ __forceinline__ bool head_of(const RopeParams &P, int pass, int sub, int &what, int &head) {
    constexpr int kHeads = 512 / D;
    const int passes_q = (P.Hq + kHeads - 1) / kHeads;
    what = pass >= passes_q, head = (pass - (what ? passes_q : 0)) * kHeads + sub;
    return head < (what ? P.H - P.Hq : P.Hq);
}

constexpr int kMostPasses = 32;  // of a warp

// The heads that a warp has left out since fp32 may not hold their squares: brought to where the larger of their largest
// channel and the root of eps is between 1 and 2, by a power of two that drops out of y.  Rare, and behind the kernel's loop,
// whose registers it would take: 9472 tokens 41.1 us a call as a part of the loop, 39.4 here, 39.1 without.
template <class E, int D, bool kVec>
__device__ __noinline__ void odd_heads(const RopeParams &P, int t, int pass, uint32_t odd_passes, const float (*weights)[D]) {
    constexpr int kLanes = D / 16;
    const int lane = threadIdx.x & 31, u = lane % kLanes;
    const Runs run = runs_of<D>(P, u);
    for (; __any_sync(0xFFFFFFFFu, odd_passes != 0); pass += P.slices, odd_passes >>= 1) {
        if (!__any_sync(0xFFFFFFFFu, odd_passes & 1)) continue;
        const bool odd = odd_passes & 1;
        int what, head;
        head_of<D>(P, pass, lane / kLanes, what, head);
        const int64_t at = static_cast<int64_t>(head) * D;
        Raw<E> x, y;
        if (odd) {
            const E *p = static_cast<const E *>(P.x[what]) + t * P.x_stride[what] + at;
            load8<E, kVec>(p + run.a, x);
            load8<E, kVec>(p + run.b, y);
        }
        float2 v[4], z[4];
        float top = sqrtf(P.eps);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[i] = odd ? make_float2(wide(x.e[2 * i]), wide(x.e[2 * i + 1])) : make_float2(0.f, 0.f);
            z[i] = odd ? make_float2(wide(y.e[2 * i]), wide(y.e[2 * i + 1])) : make_float2(0.f, 0.f);
            top = fmaxf(fmaxf(top, fmaxf(fabsf(v[i].x), fabsf(v[i].y))), fmaxf(fabsf(z[i].x), fabsf(z[i].y)));
        }
#pragma unroll
        for (int o = 1; o < kLanes; o <<= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
        // (127 + the exponent of 1 / top, so that this is a normal number)
        const int e = min(max(254 - static_cast<int>(__float_as_uint(top) >> 23), 1), 253);
        const float by = __uint_as_float(static_cast<uint32_t>(e) << 23);
        const float2 by2 = make_float2(by, by);
        float2 sum2 = make_float2(0.f, 0.f);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[i] = mul2(v[i], by2), z[i] = mul2(z[i], by2);
            sum2 = fma2(v[i], v[i], fma2(z[i], z[i], sum2));
        }
        float sum = sum2.x + sum2.y;
#pragma unroll
        for (int o = 1; o < kLanes; o <<= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
        const float r = rsqrtf(sum * (1.f / D) + P.eps * by * by);
        const float *w = weights[what];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[i] = mul2(v[i], make_float2(r * w[run.a + 2 * i], r * w[run.a + 2 * i + 1]));
            z[i] = mul2(z[i], make_float2(r * w[run.b + 2 * i], r * w[run.b + 2 * i + 1]));
        }
        if (!odd) continue;
        if (run.turned) turn(P, turns_of(P, t, u), v, z);
        E *p = static_cast<E *>(P.y[what]) + t * P.y_stride[what] + at;
        store8<E, kVec>(p + run.a, v);
        store8<E, kVec>(p + run.b, z);
    }
}

template <class E, int D, bool kVec>
__global__ void __launch_bounds__(kRopeThreads, kRopeBlocks) rope_kernel(const __grid_constant__ RopeParams P) {
    constexpr int kLanes = D / 16;       // of a head
    constexpr int kHeads = 32 / kLanes;  // of one pass
    const int lane = threadIdx.x & 31, sub = lane / kLanes, u = lane % kLanes;
    __shared__ alignas(16) float weights[2][D];
    if (P.w[0]) {
        for (int i = threadIdx.x; i < 2 * D; i += kRopeThreads) weights[i / D][i % D] = __ldg(P.w[i / D] + i % D);
        __syncthreads();
    }
    const int64_t unit = (static_cast<int64_t>(blockIdx.x) * kRopeThreads + threadIdx.x) >> 5;
    if (unit >= P.units) return;
    const int t = static_cast<int>(unit / P.slices), slice = static_cast<int>(unit - static_cast<int64_t>(t) * P.slices);

    const Runs run = runs_of<D>(P, u);
    const bool turned = run.turned;
    const int a = run.a, b = run.b;
    const int passes_q = (P.Hq + kHeads - 1) / kHeads, passes = passes_q + (P.H - P.Hq + kHeads - 1) / kHeads;
    uint32_t odd_passes = 0, this_pass = 1;  // passes in which the lane's head is one for odd_heads; at most kMostPasses
    struct {
        Raw<E> x, y;
    } next;  // the next pass, on its way
    auto fetch = [&](int pass) {
        const int what = pass >= passes_q, head = (pass - (what ? passes_q : 0)) * kHeads + sub;
        if (pass < passes && head < (what ? P.H - P.Hq : P.Hq)) {
            const E *p = static_cast<const E *>(P.x[what]) + t * P.x_stride[what] + static_cast<int64_t>(head) * D;
            load8<E, kVec>(p + a, next.x);
            load8<E, kVec>(p + b, next.y);
        }
    };
    fetch(slice);
    Turns turns;
    if (turned) turns = turns_of(P, t, u);
#pragma unroll 1
    for (int pass = slice; pass < passes; pass += P.slices) {
        const int what = pass >= passes_q, head = (pass - (what ? passes_q : 0)) * kHeads + sub;
        const bool there = head < (what ? P.H - P.Hq : P.Hq);
        float2 v[4], z[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[i] = there ? make_float2(wide(next.x.e[2 * i]), wide(next.x.e[2 * i + 1])) : make_float2(0.f, 0.f);
            z[i] = there ? make_float2(wide(next.y.e[2 * i]), wide(next.y.e[2 * i + 1])) : make_float2(0.f, 0.f);
        }
        fetch(pass + P.slices);
        bool odd = false;  // squares that fp32 may not hold
        if (P.w[0]) {
            float2 sum2 = make_float2(0.f, 0.f);
#pragma unroll
            for (int i = 0; i < 4; ++i) sum2 = fma2(v[i], v[i], fma2(z[i], z[i], sum2));
            float sum = sum2.x + sum2.y;
#pragma unroll
            for (int o = 1; o < kLanes; o <<= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
            const float mean = sum * (1.f / D) + P.eps;  // (next to a larger eps small squares do not count)
            odd = there && !(mean >= 0x1p-80f && mean <= 0x1p120f);
            odd_passes |= odd ? this_pass : 0u;
            this_pass <<= 1;
            const float r = rsqrtf(mean);
            const float2 r2 = make_float2(r, r);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const float4 p = *reinterpret_cast<const float4 *>(&weights[what][a + 4 * i]);
                const float4 q = *reinterpret_cast<const float4 *>(&weights[what][b + 4 * i]);
                v[2 * i] = mul2(v[2 * i], mul2(r2, make_float2(p.x, p.y)));
                v[2 * i + 1] = mul2(v[2 * i + 1], mul2(r2, make_float2(p.z, p.w)));
                z[2 * i] = mul2(z[2 * i], mul2(r2, make_float2(q.x, q.y)));
                z[2 * i + 1] = mul2(z[2 * i + 1], mul2(r2, make_float2(q.z, q.w)));
            }
        }
        if (turned) turn(P, turns, v, z);
        if (there && !odd) {
            E *p = static_cast<E *>(P.y[what]) + t * P.y_stride[what] + static_cast<int64_t>(head) * D;
            store8<E, kVec>(p + a, v);
            store8<E, kVec>(p + b, z);
        }
    }
    if (__any_sync(0xFFFFFFFFu, odd_passes != 0)) odd_heads<E, D, kVec>(P, t, slice, odd_passes, weights);
}

template <class E, int D>
int rope_launch(const RopeParams &P, bool vec, cudaStream_t stream) {
    const int64_t blocks = (P.units * 32 + kRopeThreads - 1) / kRopeThreads;
    if (blocks > 0x7FFFFFFF) return SSD_ERR_UNSUPPORTED;
    if (vec)
        rope_kernel<E, D, true><<<static_cast<unsigned>(blocks), kRopeThreads, 0, stream>>>(P);
    else
        rope_kernel<E, D, false><<<static_cast<unsigned>(blocks), kRopeThreads, 0, stream>>>(P);
    return launched();
}

}  // namespace
}  // namespace ssd

extern "C" int ssd_qk_rope(const void *q, const void *k, int dtype, int64_t q_stride, int64_t k_stride, int T, int Hq,
                           int Hkv, int D, const float *q_weight, const float *k_weight, float eps,
                           const int32_t *positions, const uint64_t *turns, int rot, int interleaved, void *q_out,
                           void *k_out, int64_t q_out_stride, int64_t k_out_stride, void *stream) {
    using namespace ssd;
    if (dtype != SSD_F32 && dtype != SSD_BF16 && dtype != SSD_F16) return SSD_ERR_DTYPE;
    if (T < 0 || Hq < 1 || Hkv < 1 || (D != 64 && D != 128) || rot < 0 || rot > D || rot % 16 != 0) return SSD_ERR_INVALID_ARG;
    if ((q_weight == nullptr) != (k_weight == nullptr)) return SSD_ERR_INVALID_ARG;
    if (q_weight && !(eps >= 0.f && eps <= 3.402823466e38f)) return SSD_ERR_INVALID_ARG;
    if (T > 0 && (!q || !k || !q_out || !k_out || (rot > 0 && (!positions || !turns)))) return SSD_ERR_INVALID_ARG;
    const int64_t q_row = static_cast<int64_t>(Hq) * D, k_row = static_cast<int64_t>(Hkv) * D;
    if (T > 1 && (q_stride < q_row || q_out_stride < q_row || k_stride < k_row || k_out_stride < k_row)) return SSD_ERR_INVALID_ARG;
    if (Hq > 0x7FFFFFFF / D - Hkv) return SSD_ERR_UNSUPPORTED;
    if (T == 0) return SSD_OK;
    RopeParams P{};
    P.x[0] = q, P.x[1] = k, P.y[0] = q_out, P.y[1] = k_out;
    P.x_stride[0] = q_stride, P.x_stride[1] = k_stride, P.y_stride[0] = q_out_stride, P.y_stride[1] = k_out_stride;
    P.w[0] = q_weight, P.w[1] = k_weight;
    P.positions = positions, P.turns = turns;
    P.T = T, P.Hq = Hq, P.H = Hq + Hkv;
    P.R = rot / 2, P.interleaved = interleaved != 0, P.eps = eps;
    const int heads = 512 / D, passes = (Hq + heads - 1) / heads + (Hkv + heads - 1) / heads;
    // Warps that share a token: enough that every SM has 32 (its 24 and a few to follow).  Measured with
    // 8, 16, 32 and 64 wanted: 1024 tokens 13.4, 13.4, 15.5 and 15.5 us, 9472 in bf16 38, 38, 38 and 40,
    // 4736 in fp32 40, 41, 36 and 38.
    P.slices = 1;
    while (P.slices < passes && static_cast<int64_t>(T) * P.slices < 32 * 152) P.slices *= 2;
    if (P.slices > passes) P.slices = passes;
    // (a warp has no more passes than it has marks for)
    if (P.slices < (passes + kMostPasses - 1) / kMostPasses) P.slices = (passes + kMostPasses - 1) / kMostPasses;
    P.units = static_cast<int64_t>(T) * P.slices;
    const int es = dtype == SSD_F32 ? 4 : 2;
    const bool vec = aligned(q, 16) && aligned(k, 16) && aligned(q_out, 16) && aligned(k_out, 16) && q_stride * es % 16 == 0 &&
                     k_stride * es % 16 == 0 && q_out_stride * es % 16 == 0 && k_out_stride * es % 16 == 0;
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (dtype == SSD_F32) return D == 64 ? rope_launch<float, 64>(P, vec, s) : rope_launch<float, 128>(P, vec, s);
    if (dtype == SSD_BF16)
        return D == 64 ? rope_launch<__nv_bfloat16, 64>(P, vec, s) : rope_launch<__nv_bfloat16, 128>(P, vec, s);
    return D == 64 ? rope_launch<__half, 64>(P, vec, s) : rope_launch<__half, 128>(P, vec, s);
}
