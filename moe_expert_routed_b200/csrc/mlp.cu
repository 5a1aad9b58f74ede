// mlp.cu -- the gated expert MLP of a layer (include/moe_qmm.h, moe_mlp):
//   h[t][s]  = act(G_e x_t) * (U_e x_t),        e = ids[t][s]
//   out[t]   = residual[t] + sum_s weights[t][s] * (D_e h[t][s])
// Three ways, chosen by size:
//   few tokens   the two kernels of mlp_few.cu (the sum over the slots happens in
//                the down projection's kernel);
//   up to some tens of pairs an expert, 16-bit types
//                the grouped products of mlp_mid.cu and the weighted sum;
//   otherwise    the fused gate+up product, the down product over the pairs and the
//                weighted sum, each a call of this library.
#include "common.cuh"
#include "internal.h"

namespace moe {
namespace {

inline size_t al256(size_t v) { return (v + 255) & ~(size_t)255; }

// Type of h between the two products. bf16 x and a bf16 result: bf16, the rounding every
// bf16 model makes there (it adds 2^-9 of each h once, next to the 2^-9 of the result's own
// rounding, and has f32's range). Otherwise f32: |h| can leave f16's range (two factors),
// and bf16 would cost an f16 result 3 of its bits and an f32 result 7 more of those that
// the split of f32 operands into two bf16 terms leaves (16).
moe_dtype h_dtype(int x_dtype, int out_dtype) {
    return x_dtype == DT_BF16 && out_dtype == DT_BF16 ? MOE_BF16 : MOE_F32;
}

struct Layout {
    size_t own, h, z, total;  // own: workspace of the products, at offset 0 (the error word first)
};

bool layout(uint32_t m, uint32_t hidden, uint32_t inter, uint32_t S, uint32_t E, int x_dtype, Layout *L) {
    const uint64_t R = (uint64_t)m * S;
    if (R > 0x7FFFFFFFull) return false;
    const uint64_t few = mlp_few_workspace(m, hidden, inter, S);
    const size_t a = moe_qmm_id_workspace_bytes_k(m, hidden, S, E, (moe_dtype)x_dtype);
    // whatever the result's type, with room for either type of h
    const size_t b = moe_qmm_id_workspace_bytes_k((uint32_t)R, inter, 1, E, MOE_F32);
    const size_t c = x_dtype == DT_BF16 ? moe_qmm_id_workspace_bytes_k((uint32_t)R, inter, 1, E, MOE_BF16) : b;
    if (!a || !b || !c) return false;
    L->own = al256(tmax(a, tmax(b, c)));
    L->h = L->own;
    L->z = L->h + al256(R * inter * 4ull);
    L->total = L->z + al256(R * hidden * 4ull);
    // the few-token kernels' planes of h take the same room
    const uint64_t mid = mlp_mid_workspace(m, hidden, inter, S, E);
    if (L->total < L->h + al256(few)) L->total = L->h + al256(few);
    if (L->total < L->h + al256(mid)) L->total = L->h + al256(mid);
    return true;
}

moe_status check_weights(const moe_expert_weights *w, uint32_t k, uint32_t n) {
    if (!w) return MOE_ERR_INVALID_ARGUMENT;
    if (w->bias && ((int)w->bias_dtype < 0 || (int)w->bias_dtype > 2)) return MOE_ERR_INVALID_ARGUMENT;
    // sizes, formats and pointers by the rules of the product itself
    return validate_call(w->packed, (const uint32_t *)w->packed, w->packed, w->scales, w->aux, w->packed, 1, k, n,
                         w->group_size, w->bits, w->fmt, 1, 1, MOE_F32, MOE_F32);
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" {

size_t moe_mlp_workspace_bytes(uint32_t m, uint32_t hidden, uint32_t inter, uint32_t n_expert_used,
                               uint32_t num_experts, moe_dtype x_dtype) {
    Layout L;
    if (!m || !hidden || !inter || !n_expert_used || !num_experts || (int)x_dtype < 0 || (int)x_dtype > 2) return 0;
    return layout(m, hidden, inter, n_expert_used, num_experts, (int)x_dtype, &L) ? L.total : 0;
}

moe_status moe_mlp(const void *x, const uint32_t *ids, const float *weights, const moe_expert_weights *gate_up,
                   const moe_expert_weights *down, const void *residual, void *out, uint32_t m, uint32_t hidden,
                   uint32_t inter, uint32_t n_expert_used, uint32_t num_experts, moe_dtype x_dtype,
                   moe_dtype out_dtype, moe_act act, void *workspace, size_t workspace_bytes, moe_path path,
                   moe_stream_t stream) {
    if (!m || !hidden || !inter || !n_expert_used || !num_experts || inter > 0x7FFFFFFFu)
        return MOE_ERR_INVALID_ARGUMENT;
    if ((int)x_dtype < 0 || (int)x_dtype > 2 || (int)out_dtype < 0 || (int)out_dtype > 2 || (int)act < 0 ||
        (int)act > 2 || (int)path < 0 || (int)path > 2)
        return MOE_ERR_INVALID_ARGUMENT;
    if (!x || !ids || !weights || !out) return MOE_ERR_INVALID_ARGUMENT;
    moe_status v = check_weights(gate_up, hidden, 2u * inter);
    if (v == MOE_OK) v = check_weights(down, inter, hidden);
    if (v != MOE_OK) return v;
    const uintptr_t xm = x_dtype == MOE_F32 ? 3u : 1u, om = out_dtype == MOE_F32 ? 3u : 1u;
    if (((uintptr_t)x & xm) || (((uintptr_t)out | (uintptr_t)residual) & om) ||
        (((uintptr_t)ids | (uintptr_t)weights) & 3u) || !workspace || ((uintptr_t)workspace & 15u))
        return MOE_ERR_INVALID_ARGUMENT;
    Layout L;
    if (!layout(m, hidden, inter, n_expert_used, num_experts, (int)x_dtype, &L)) return MOE_ERR_UNSUPPORTED;
    if (workspace_bytes < L.total) return MOE_ERR_WORKSPACE_TOO_SMALL;

    uint8_t *ws = (uint8_t *)workspace;
    const uint32_t R = m * n_expert_used;
    void *h = ws + L.h, *z = ws + L.z;
    const MlpArgs a{x,      ids,   weights, gate_up,       down,        residual,     out,           m,
                    hidden, inter, n_expert_used, num_experts, (int)x_dtype, (int)out_dtype, (int)act};
    // The few-token kernels have four pairs' worth of tensor work for one and no routing;
    // mlp_mid.cu's products route first, then read and expand an expert's weights once for 24
    // pairs, and gain the more, the longer that takes. Few against mid, 2,816 x 704
    // experts, us: 256 experts at 1/2 pair an expert 101 / 135 (affine 4 bits), 103 / 116 (NVFP4),
    // 204 / 192 (3-bit codebook), 221 / 157 (affine 8 bits); at 1 pair 184 / 199, 193 / 172, 376 /
    // 292, 391 / 232; at 2 pairs 288 / 261, 313 / 227, 531 / 390, 604 / 306. Of 8 experts, 16 pairs
    // in all 23 / 33, 23 / 29, 38 / 40, 40 / 39; 32 pairs 40 / 34, 42 / 32, 48 / 40, 53 / 40.
    // (The codebooks of 2 and 4 bits and 6-bit codes follow the 3-bit codebook, MXFP4 follows
    // NVFP4, by likeness.) Where mlp_mid.cu does not apply (32-bit types) the grouped products are left: few
    // against grouped, 16-bit types, at 4 pairs an expert 110 / 177 (affine 4 bits), 116 / 128
    // (NVFP4), 147 / 180 (affine 8 bits), at 8 171 / 179, 179 / 131, 268 / 183; 64 pairs of 8
    // experts 49 / 79, 52 / 63, 66 / 83.
    const bool mid = path == MOE_PATH_AUTO && mlp_mid_supported(a);
    auto narrow = [](const moe_expert_weights *w) { return w->bits == 4 && w->fmt != MOE_FMT_CODEBOOK; };
    const uint64_t few_to = !mid ? tmax<uint64_t>(64u, 4ull * num_experts)
                                 : tmax<uint64_t>(16u, narrow(gate_up) && narrow(down) ? num_experts : num_experts / 4u);
    if (path != MOE_PATH_GROUPED && (path == MOE_PATH_DECODE || R <= few_to) && mlp_few_supported(a))
        return status_of(launch_mlp_few(a, (uint32_t *)ws, h, (cudaStream_t)stream));
    if (mid) return status_of(launch_mlp_mid(a, ws, ws + L.h, (cudaStream_t)stream));
    const moe_dtype hd = h_dtype((int)x_dtype, (int)out_dtype);
    LayerProduct layer{0u};
    v = run_product(x, ids, *gate_up, h, m, hidden, 2u * inter, n_expert_used, num_experts, x_dtype, hd, (int)act,
                    workspace, L.own, stream, path, &layer);
    if (v != MOE_OK) return v;
    // every (token, slot) pair is a token of its own here, with its own row of h; pairs
    // left out have no row of z
    v = run_product(h, ids, *down, z, R, inter, hidden, 1, num_experts, hd, MOE_F32, -1, workspace, L.own, stream, path,
                    &layer);
    if (v != MOE_OK) return v;
    return status_of(launch_combine(z, weights, ids, residual, out, m, n_expert_used, hidden, num_experts, DT_F32,
                                    (int)out_dtype, (cudaStream_t)stream));
}

}  // extern "C"
