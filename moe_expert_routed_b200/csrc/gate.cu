// gate.cu -- the router's choice: the top-k experts of each token from its
// logits, and their weights (include/moe_qmm.h, moe_gate_topk).
//
// One warp per token. Lane l holds logits l, l + 32, ... in registers as keys
// whose unsigned order is the order of the choice; each of the k rounds takes the
// largest key of the warp (redux.max) and the lowest expert that has it (redux.min),
// and retires it where it is. Bound by the ALU: about five instructions a round for
// each register, so the registers are as few as the experts need. (Looking for the
// key by a vote and a branch a register took more, and longer for few tokens.)
// Softmax and sigmoid are monotonic, so without a selection bias the choice is made
// on the logits themselves and is exact. With a bias the choice is by sigmoid(l) + b:
// two experts can then lie closer than a 32-bit sigmoid tells apart, so that sum is
// formed in 64 bits and compared as a 64-bit key (two redux rounds).
#include "common.cuh"
#include "internal.h"

namespace moe {
namespace {

constexpr int GATE_WARPS = 4;  // tokens per CTA
constexpr uint32_t FULL = 0xFFFFFFFFu;

// Keys: 0 retired or no expert, 1 NaN (below every number), else increasing with v.
__device__ __forceinline__ uint32_t key32(float v) {
    if (v != v) return 1u;
    const uint32_t u = __float_as_uint(v + 0.f);  // -0 and +0 tie
    return (u & 0x80000000u) ? ~u : u | 0x80000000u;
}

__device__ __forceinline__ uint64_t key64(double v) {
    if (v != v) return 1ull;
    const uint64_t u = (uint64_t)__double_as_longlong(v + 0.0);
    return (u >> 63) ? ~u : u | (1ull << 63);
}

struct GateParams {
    const void *logits;
    const float *bias;
    uint32_t *ids;
    float *weights;
    uint32_t m, E, k;
    int dtype, sigmoid, renorm;
    float scale;
};

// V: logits per lane (E <= 32 V). BIAS: sigmoid scores chosen with a selection bias.
template <int V, bool BIAS>
__global__ void __launch_bounds__(GATE_WARPS * 32) gate_topk(const GateParams P) {
    const uint32_t lane = threadIdx.x & 31u;
    const uint64_t t = (uint64_t)blockIdx.x * GATE_WARPS + (threadIdx.x >> 5);
    if (t >= P.m) return;
    const size_t row = t * P.E;
    float l[V];
    uint32_t hi[V], lo[BIAS ? V : 1];
#pragma unroll
    for (int j = 0; j < V; j++) {
        const uint32_t e = j * 32u + lane;
        l[j] = e < P.E ? load_x(P.logits, P.dtype, row + e) : 0.f;
    }
#pragma unroll
    for (int j = 0; j < V; j++) {
        const uint32_t e = j * 32u + lane;
        if constexpr (BIAS) {
            const uint64_t key =
                e < P.E ? key64(1.0 / (1.0 + exp(-(double)l[j])) + (double)__ldg(P.bias + e)) : 0ull;
            hi[j] = (uint32_t)(key >> 32);
            lo[j] = (uint32_t)key;
        } else {
            hi[j] = e < P.E ? key32(l[j]) : 0u;
        }
    }

    // rounds: lane r keeps the r-th choice (k <= 32 and k <= E: a key above 0 is left)
    uint32_t my_e = 0;
    for (uint32_t r = 0; r < P.k; r++) {
        uint32_t top = 0, low = 0;
        if constexpr (BIAS) {
#pragma unroll
            for (int j = 0; j < V; j++)
                if (hi[j] > top || (hi[j] == top && lo[j] > low)) top = hi[j], low = lo[j];
            const uint32_t w = __reduce_max_sync(FULL, top);
            low = __reduce_max_sync(FULL, top == w ? low : 0u);
            top = w;
        } else {
#pragma unroll
            for (int j = 0; j < V; j++) top = max(top, hi[j]);
            top = __reduce_max_sync(FULL, top);
        }
        uint32_t slot = FULL;  // the lowest register of this lane that has it
#pragma unroll
        for (int j = V - 1; j >= 0; j--) {
            bool is = hi[j] == top;
            if constexpr (BIAS) is = is && lo[j] == low;
            if (is) slot = j;
        }
        const uint32_t e = __reduce_min_sync(FULL, slot == FULL ? FULL : slot * 32u + lane);
        if ((e & 31u) != lane) slot = FULL;
#pragma unroll
        for (int j = 0; j < V; j++)
            if (slot == (uint32_t)j) {
                hi[j] = 0u;
                if constexpr (BIAS) lo[j] = 0u;
            }
        if (lane == r) my_e = e;
    }

    // weights of the chosen
    const bool mine = lane < P.k;
    const float my_l = mine ? load_x(P.logits, P.dtype, row + my_e) : 0.f;
    float p = 0.f, den = 1.f;
    if (P.sigmoid) {
        // in 64 bits: far below zero a 32-bit sigmoid leaves nothing to renormalise
        double s = mine ? 1.0 / (1.0 + exp(-(double)my_l)) : 0.0;
        if (P.renorm) {
            double sum = s;
#pragma unroll
            for (int d = 16; d > 0; d >>= 1) sum += __shfl_xor_sync(FULL, sum, d);
            s = sum == 0.0 ? 0.0 : s / sum;
        }
        p = (float)s;
    } else {
        const float mx = __shfl_sync(FULL, my_l, 0);  // the first choice
        p = mine ? expf(my_l - mx) : 0.f;
        float sum = p;
        if (!P.renorm) {
            sum = 0.f;
#pragma unroll
            for (int j = 0; j < V; j++)
                if (j * 32u + lane < P.E) sum += expf(l[j] - mx);
        }
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) sum += __shfl_xor_sync(FULL, sum, d);
        den = sum;
        if (mx == -INFINITY) {  // every expert masked: weights 0, unless a NaN is among them
            bool nan = false;
#pragma unroll
            for (int j = 0; j < V; j++) nan |= l[j] != l[j];
            if (!__any_sync(FULL, nan)) p = 0.f, den = 1.f;
        }
    }
    if (mine) {
        const size_t o = t * P.k + lane;
        P.ids[o] = my_e;
        P.weights[o] = P.scale * (p / den);
    }
}

template <bool BIAS>
cudaError_t launch_v(const GateParams &P, cudaStream_t st) {
    const dim3 grid((P.m + GATE_WARPS - 1) / GATE_WARPS), block(GATE_WARPS * 32);
    switch ((P.E + 31u) / 32u) {
        case 1: gate_topk<1, BIAS><<<grid, block, 0, st>>>(P); break;
        case 2: gate_topk<2, BIAS><<<grid, block, 0, st>>>(P); break;
        case 3: gate_topk<3, BIAS><<<grid, block, 0, st>>>(P); break;
        case 4: gate_topk<4, BIAS><<<grid, block, 0, st>>>(P); break;
        case 5: gate_topk<5, BIAS><<<grid, block, 0, st>>>(P); break;
        case 6: gate_topk<6, BIAS><<<grid, block, 0, st>>>(P); break;
        case 7:
        case 8: gate_topk<8, BIAS><<<grid, block, 0, st>>>(P); break;
        default:
            if (P.E <= 384) gate_topk<12, BIAS><<<grid, block, 0, st>>>(P);
            else if (P.E <= 512) gate_topk<16, BIAS><<<grid, block, 0, st>>>(P);
            else gate_topk<32, BIAS><<<grid, block, 0, st>>>(P);
    }
    return cudaGetLastError();
}

}  // namespace
}  // namespace moe

extern "C" moe_status moe_gate_topk(const void *logits, const float *select_bias, uint32_t *ids, float *weights,
                                    uint32_t m, uint32_t num_experts, uint32_t top_k, moe_dtype logits_dtype,
                                    moe_score score, int renormalize, float scale, moe_stream_t stream) {
    if (!m || !num_experts || !top_k || top_k > num_experts) return MOE_ERR_INVALID_ARGUMENT;
    if ((int)logits_dtype < 0 || (int)logits_dtype > 2 || (int)score < 0 || (int)score > 1)
        return MOE_ERR_INVALID_ARGUMENT;
    if (!logits || !ids || !weights || (select_bias && score != MOE_SCORE_SIGMOID)) return MOE_ERR_INVALID_ARGUMENT;
    const uintptr_t la = logits_dtype == MOE_F32 ? 3u : 1u;
    if (((uintptr_t)logits & la) || (((uintptr_t)ids | (uintptr_t)weights | (uintptr_t)select_bias) & 3u))
        return MOE_ERR_INVALID_ARGUMENT;
    if (num_experts > MOE_ROUTE_MAX_EXPERTS || top_k > MOE_GATE_MAX_TOPK || m > 0x7FFFFFFFu)
        return MOE_ERR_UNSUPPORTED;
    const moe::GateParams P{logits, select_bias, ids, weights, m, num_experts, top_k, (int)logits_dtype,
                            score == MOE_SCORE_SIGMOID, renormalize != 0, scale};
    const cudaError_t ce =
        select_bias ? moe::launch_v<true>(P, (cudaStream_t)stream) : moe::launch_v<false>(P, (cudaStream_t)stream);
    return ce == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}
