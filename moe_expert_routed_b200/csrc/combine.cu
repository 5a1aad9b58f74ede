// combine.cu -- the weighted sum of a token's rows (include/moe_qmm.h, moe_combine):
//   out[t][c] = residual[t][c] + sum_s weights[t][s] * z[t][s][c]
// in one pass over z. Bound by memory: every byte of z is read once, out is
// written once. A thread owns VEC neighbouring columns of one token and walks the
// slots in order, so the sum (fp32) has one order and no atomics; the residual is
// added last, before the only rounding. Rows are requested B slots ahead without branches:
// 4,096 x 8 x 4,096 bf16 with a residual 51 us, 6.6 TB/s, against 83 one slot at a time (and
// 161 with the requests under a condition).
#include <string.h>

#include "common.cuh"
#include "internal.h"

namespace moe {
namespace {

constexpr int COMBINE_THREADS = 256;

struct CombineParams {
    const void *z;
    const float *w;  // null: 1 (rows that carry their weights)
    const uint32_t *ids;
    const void *residual;
    void *out;
    uint64_t total;  // m * (n / VEC)
    uint32_t S, n, E;
};

template <typename T> struct Cvt;
template <> struct Cvt<float> {
    static __device__ __forceinline__ float to(float v) { return v; }
    static __device__ __forceinline__ float from(float v) { return v; }
};
template <> struct Cvt<__nv_bfloat16> {
    static __device__ __forceinline__ float to(__nv_bfloat16 v) { return __bfloat162float(v); }
    static __device__ __forceinline__ __nv_bfloat16 from(float v) { return __float2bfloat16_rn(v); }
};
template <> struct Cvt<__half> {
    static __device__ __forceinline__ float to(__half v) { return __half2float(v); }
    static __device__ __forceinline__ __half from(float v) { return __float2half_rn(v); }
};

template <typename T, int N> struct alignas(sizeof(T) * N) Pack { T v[N]; };

// Read once: not kept in L1.
template <typename T, int N>
__device__ __forceinline__ Pack<T, N> load_once(const Pack<T, N> *p) {
    Pack<T, N> v;
    if constexpr (sizeof(v) == 16) {
        const uint4 u = __ldcs((const uint4 *)p);
        memcpy(&v, &u, 16);
    } else if constexpr (sizeof(v) == 8) {
        const uint2 u = __ldcs((const uint2 *)p);
        memcpy(&v, &u, 8);
    } else {
        v = *p;
    }
    return v;
}

// I: 32-bit indices where the sizes allow (the division by nv is several times cheaper).
// B > 0: the slots are a multiple of B and none is left out, so B rows are requested
// before the first is used; B = 0: one at a time.
template <typename TZ, typename TO, int VEC, int B, typename I>
__global__ void __launch_bounds__(COMBINE_THREADS) combine_kernel(const CombineParams P) {
    const I nv = P.n / VEC;
    const I i = (I)blockIdx.x * COMBINE_THREADS + threadIdx.x;
    if (i >= (I)P.total) return;
    const I t = i / nv;
    const I c = i - t * nv;
    const Pack<TZ, VEC> *z = (const Pack<TZ, VEC> *)P.z + (size_t)t * P.S * nv + c;
    const float *w = P.w + (size_t)t * P.S;
    float acc[VEC];
#pragma unroll
    for (int j = 0; j < VEC; j++) acc[j] = 0.f;
    if constexpr (B > 0) {
        for (uint32_t s0 = 0; s0 < P.S; s0 += B, z += (size_t)B * nv) {
            Pack<TZ, VEC> v[B];
#pragma unroll
            for (int k = 0; k < B; k++) v[k] = load_once(z + (size_t)k * nv);
#pragma unroll
            for (int k = 0; k < B; k++) {
                const float ws = P.w ? __ldg(w + s0 + k) : 1.f;
#pragma unroll
                for (int j = 0; j < VEC; j++) acc[j] = fmaf(ws, Cvt<TZ>::to(v[k].v[j]), acc[j]);
            }
        }
    } else {
        for (uint32_t s = 0; s < P.S; s++) {
            if (P.ids && __ldg(P.ids + (size_t)t * P.S + s) >= P.E) continue;  // not read
            const float ws = P.w ? __ldg(w + s) : 1.f;
            const Pack<TZ, VEC> v = load_once(z + (size_t)s * nv);
#pragma unroll
            for (int j = 0; j < VEC; j++) acc[j] = fmaf(ws, Cvt<TZ>::to(v.v[j]), acc[j]);
        }
    }
    Pack<TO, VEC> o;
    if (P.residual) {
        const Pack<TO, VEC> r = ((const Pack<TO, VEC> *)P.residual)[i];
#pragma unroll
        for (int j = 0; j < VEC; j++) acc[j] += Cvt<TO>::to(r.v[j]);
    }
#pragma unroll
    for (int j = 0; j < VEC; j++) o.v[j] = Cvt<TO>::from(acc[j]);
    ((Pack<TO, VEC> *)P.out)[i] = o;
}

template <typename TZ, typename TO, int VEC, int B>
cudaError_t launch_b(CombineParams P, uint64_t m, cudaStream_t st) {
    P.total = m * (P.n / VEC);
    const uint64_t blocks = (P.total + COMBINE_THREADS - 1) / COMBINE_THREADS;
    if (blocks > 0x7FFFFFFFull) return cudaErrorInvalidConfiguration;
    if (blocks * COMBINE_THREADS <= 0xFFFFFFFFull)
        combine_kernel<TZ, TO, VEC, B, uint32_t><<<(uint32_t)blocks, COMBINE_THREADS, 0, st>>>(P);
    else
        combine_kernel<TZ, TO, VEC, B, uint64_t><<<(uint32_t)blocks, COMBINE_THREADS, 0, st>>>(P);
    return cudaGetLastError();
}

template <typename TZ, typename TO, int VEC>
cudaError_t launch_v(const CombineParams &P, uint64_t m, cudaStream_t st) {
    if (P.ids || P.S % 2u) return launch_b<TZ, TO, VEC, 0>(P, m, st);
    return P.S % 4u ? launch_b<TZ, TO, VEC, 2>(P, m, st) : launch_b<TZ, TO, VEC, 4>(P, m, st);
}

template <typename TZ, typename TO>
cudaError_t launch_t(const CombineParams &P, uint64_t m, cudaStream_t st) {
    // 16 bytes of z an access where rows start and end on their boundaries, single elements elsewhere
    constexpr int W = 16 / sizeof(TZ);
    const uintptr_t za = (uintptr_t)P.z, oa = (uintptr_t)P.out | (uintptr_t)P.residual;
    if (P.n % W == 0 && za % (W * sizeof(TZ)) == 0 && oa % (W * sizeof(TO)) == 0)
        return launch_v<TZ, TO, W>(P, m, st);
    return launch_v<TZ, TO, 1>(P, m, st);
}

template <typename TZ>
cudaError_t launch_z(const CombineParams &P, uint64_t m, int out_dtype, cudaStream_t st) {
    if (out_dtype == DT_F32) return launch_t<TZ, float>(P, m, st);
    if (out_dtype == DT_BF16) return launch_t<TZ, __nv_bfloat16>(P, m, st);
    return launch_t<TZ, __half>(P, m, st);
}

}  // namespace

cudaError_t launch_combine(const void *z, const float *weights, const uint32_t *ids, const void *residual, void *out,
                           uint32_t m, uint32_t S, uint32_t n, uint32_t E, int z_dtype, int out_dtype,
                           cudaStream_t st) {
    const CombineParams P{z, weights, ids, residual, out, 0, S, n, E};
    if (z_dtype == DT_F32) return launch_z<float>(P, m, out_dtype, st);
    if (z_dtype == DT_BF16) return launch_z<__nv_bfloat16>(P, m, out_dtype, st);
    return launch_z<__half>(P, m, out_dtype, st);
}

}  // namespace moe

extern "C" moe_status moe_combine(const void *z, const float *weights, const uint32_t *ids, const void *residual,
                                  void *out, uint32_t m, uint32_t n_expert_used, uint32_t n, uint32_t num_experts,
                                  moe_dtype z_dtype, moe_dtype out_dtype, moe_stream_t stream) {
    if (!m || !n_expert_used || !n || (ids && !num_experts)) return MOE_ERR_INVALID_ARGUMENT;
    if ((int)z_dtype < 0 || (int)z_dtype > 2 || (int)out_dtype < 0 || (int)out_dtype > 2)
        return MOE_ERR_INVALID_ARGUMENT;
    if (!z || !weights || !out) return MOE_ERR_INVALID_ARGUMENT;
    const uintptr_t zm = z_dtype == MOE_F32 ? 3u : 1u, om = out_dtype == MOE_F32 ? 3u : 1u;
    if (((uintptr_t)z & zm) || (((uintptr_t)out | (uintptr_t)residual) & om) ||
        (((uintptr_t)weights | (uintptr_t)ids) & 3u))
        return MOE_ERR_INVALID_ARGUMENT;
    if ((uint64_t)m * n_expert_used > 0x7FFFFFFFull) return MOE_ERR_UNSUPPORTED;
    return moe::status_of(moe::launch_combine(z, weights, ids, residual, out, m, n_expert_used, n, num_experts,
                                              (int)z_dtype, (int)out_dtype, (cudaStream_t)stream));
}
