// gate.cu -- the router's choice: the top-k experts of each token from its
// logits, and their weights (include/moe_qmm.h, moe_gate_topk).
//
// One warp per token. Lane l holds logits l, l + 32, ... in registers as keys
// whose unsigned order is the order of the choice; each of the k rounds takes the
// largest key of the warp (redux.max) and the lowest expert that has it (redux.min),
// and retires it where it is. Bound by the ALU: about five instructions a round for
// each register, so the registers are as few as the experts need. (Looking for the
// key by a vote and a branch a register took more, and longer for few tokens.)
// 8,192 x 256 f32 logits, top-8: 8.7 us on the device (floor 1.4, their bytes); 1 x 128: 2.1.
// Softmax and sigmoid are monotonic, so without a selection bias the choice is made
// on the logits themselves and is exact. With a bias the choice is by sigmoid(l) + b:
// two experts can then lie closer than a 32-bit sigmoid tells apart, so that sum is
// formed in 64 bits and compared as a 64-bit key (two redux rounds). The 64-bit
// exponentials would bound it (8,192 x 256: 23 us against 17; 257 x 160: 6.5), so they are taken only of the
// experts that a 32-bit score with its error bound cannot rule out: as a rule the k
// chosen and few more, one a lane.
#include "common.cuh"
#include "internal.h"

namespace moe {
namespace {

constexpr int GATE_WARPS = 4;  // tokens per CTA
constexpr uint32_t FULL = 0xFFFFFFFFu;

// Keys: 0 retired or no expert, 1 NaN (below every number), 2 an expert masked by a logit of
// -inf under a selection bias (below every score, whatever the bias: the bias is not added),
// else increasing with v. Without a bias the logit -inf is the lowest number by itself.
constexpr uint32_t MASKED = 2u;
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

// sigmoid(l) + b in 64 bits, as a key.
__device__ __forceinline__ uint64_t biased_key(float l, float b) {
    return l == -INFINITY ? (uint64_t)MASKED : key64(1.0 / (1.0 + exp(-(double)l)) + (double)b);
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

// The choice among all experts: lane r's my_e is the r-th.
template <int V, bool BIAS>
__device__ __forceinline__ void choose(const GateParams &P, const float (&l)[V], uint32_t lane, uint32_t &my_e) {
    uint32_t hi[V], lo[BIAS ? V : 1];
#pragma unroll
    for (int j = 0; j < V; j++) {
        const uint32_t e = j * 32u + lane;
        if constexpr (BIAS) {
            const uint64_t key = e < P.E ? biased_key(l[j], __ldg(P.bias + e)) : 0ull;
            hi[j] = (uint32_t)(key >> 32);
            lo[j] = (uint32_t)key;
        } else {
            hi[j] = e < P.E ? key32(l[j]) : 0u;
        }
    }

    // rounds: lane r keeps the r-th choice (k <= 32 and k <= E: a key above 0 is left)
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
}

// The same with a selection bias, among the experts whose 32-bit score may reach the k-th:
// false if there are more than 32 of those. The score is off by less than 2^-21: of the
// sigmoid s, s (1 - s) (2 + 1.16 |l|) 2^-23 < 1.3 * 2^-24 by __expf (its largest value is near
// |l| = 0.8), 2^-24 by the sum, 2^-22 by __fdividef (2 units in the last place); and 2^-24
// of the sum with the bias. Twice that is allowed for. An expert among the k best scores no less than the k-th largest lower
// bound, so its upper bound does not lie below that.
template <int V>
__device__ __forceinline__ bool choose_few(const GateParams &P, const float (&l)[V], size_t row, uint32_t *few,
                                           uint32_t lane, uint32_t &my_e) {
    float v[V];
    uint32_t low[V];
#pragma unroll
    for (int j = 0; j < V; j++) {
        const uint32_t e = j * 32u + lane;
        v[j] = e < P.E ? __fdividef(1.f, 1.f + __expf(-l[j])) + __ldg(P.bias + e) : 0.f;
        const float d = isinf(v[j]) ? 0.f : fmaf(fabsf(v[j]), 0x1p-23f, 0x1p-20f);
        low[j] = e >= P.E ? 0u : l[j] == -INFINITY ? MASKED : key32(v[j] - d);
    }
    uint32_t cut = 0, n = 0;
    while (n < P.k) {  // takes away all that are as large as the largest left; k <= E
        uint32_t top = 0, same = 0;
#pragma unroll
        for (int j = 0; j < V; j++) top = max(top, low[j]);
        cut = __reduce_max_sync(FULL, top);
#pragma unroll
        for (int j = 0; j < V; j++)
            if (low[j] == cut) low[j] = 0u, same++;
        n += __reduce_add_sync(FULL, same);
    }
    uint32_t c = 0;
#pragma unroll
    for (int j = 0; j < V; j++) {
        const uint32_t e = j * 32u + lane;
        const float d = isinf(v[j]) ? 0.f : fmaf(fabsf(v[j]), 0x1p-23f, 0x1p-20f);
        const bool in = e < P.E && (l[j] == -INFINITY ? MASKED : key32(v[j] + d)) >= cut;
        const uint32_t who = __ballot_sync(FULL, in), at = c + __popc(who & ((1u << lane) - 1u));
        if (in && at < 32u) few[at] = e;
        c += __popc(who);
    }
    if (c > 32u) return false;
    __syncwarp();
    // one a lane, by expert
    uint32_t hi = 0u, lo = 0u, mine = 0u;
    if (lane < c) {
        mine = few[lane];
        const float x = load_x(P.logits, P.dtype, row + mine);
        const uint64_t key = biased_key(x, __ldg(P.bias + mine));
        hi = (uint32_t)(key >> 32);
        lo = (uint32_t)key;
    }
    for (uint32_t r = 0; r < P.k; r++) {
        const uint32_t top = __reduce_max_sync(FULL, hi), low32 = __reduce_max_sync(FULL, hi == top ? lo : 0u);
        const uint32_t first = __ffs(__ballot_sync(FULL, lane < c && hi == top && lo == low32)) - 1u;
        const uint32_t e = __shfl_sync(FULL, mine, first);
        if (lane == r) my_e = e;
        if (lane == first) hi = lo = 0u;
    }
    return true;
}

// V: logits per lane (E <= 32 V). BIAS: sigmoid scores chosen with a selection bias.
template <int V, bool BIAS>
__global__ void __launch_bounds__(GATE_WARPS * 32) gate_topk(const GateParams P) {
    const uint32_t lane = threadIdx.x & 31u;
    const uint64_t t = (uint64_t)blockIdx.x * GATE_WARPS + (threadIdx.x >> 5);
    if (t >= P.m) return;
    const size_t row = t * P.E;
    float l[V];
#pragma unroll
    for (int j = 0; j < V; j++) {
        const uint32_t e = j * 32u + lane;
        l[j] = e < P.E ? load_x(P.logits, P.dtype, row + e) : 0.f;
    }
    uint32_t my_e = 0;
    bool done = false;
    if constexpr (BIAS) {
        __shared__ uint32_t few[GATE_WARPS][32];
        done = choose_few<V>(P, l, row, few[threadIdx.x >> 5], lane, my_e);
    }
    if (!done) choose<V, BIAS>(P, l, lane, my_e);

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
    return moe::status_of(select_bias ? moe::launch_v<true>(P, (cudaStream_t)stream)
                                      : moe::launch_v<false>(P, (cudaStream_t)stream));
}
