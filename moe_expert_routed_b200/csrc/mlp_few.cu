// mlp_few.cu -- the gated expert MLP for few tokens, in two kernels: what a decode
// step of one or a few sequences runs.
//
//   mlp_up    h[p] = act(G_e x_t) * (U_e x_t), times the pair's weight (and, NVFP4, the
//             down projection's scale2), split into planes in the workspace
//   mlp_down  out[t] = residual[t] + sum over the token's pairs of D_e h[p]
//
// Both are bound by the bytes of the weights that the tokens' experts hold, so each
// row of codes is read once for all pairs of its expert (up to the pairs of a pass),
// straight from global memory into the lane that needs it, several steps ahead
// (cp.async into a ring that belongs to the lane: no barrier in the loop).
//
// The arithmetic must not become the bound instead. It runs on mma.sync m16n8k16 with
// f16 operands and f32 sums: a tile is 16 weight rows, the eight columns are x.
//   A 4-bit integer code c masked out of its word is the f16 subnormal c 2^-24 (or c
// 2^-20 one nibble higher, which x makes up for): eight codes take five logic
// operations. E2M1 codes go through the hardware's conversion, four operations. Both
// are exact. Measured per 8-code word and scheduler, MMA included: 13.5 and 11
// cycles, against 26 to bf16 operands and 26 for E2M1 by shifts; E4M3 operands are
// converted to f16 before the legacy MMA anyway and took twice the instructions.
//   x and h enter as f16 planes: a unit of 32 values is scaled by a power of two to below
// 2^15, the first plane is its rounding to f16, the second that of the remainder. One
// plane holds bf16 and f16 x exactly (down to 2^-38 of the unit's largest value); f32 x
// takes two, 22 bits. h, the f32 result of mlp_up, takes one for a bf16 result (11
// bits, 3 more than the rounding to bf16 that the result gets anyway) and two otherwise.
//   Scales of weights and of x are applied to f32 sums of one unit. The four lanes
// that share a row each hold another unit (their 16-byte load), so a column belongs to
// one unit: lane q's x stands in column q, the other lanes are zero there, and the
// accumulator keeps the four units apart in four columns; the eight columns hold two
// sets (two pairs, or the two planes of one pair).
// tcgen05's 128-row tiles with one or two columns in use would waste more than this
// does, and need their operand in shared or tensor memory.
#include "common.cuh"
#include "internal.h"
#include "ptx.cuh"

namespace moe {
namespace {

constexpr uint32_t FULL = 0xFFFFFFFFu;
constexpr uint32_t FEW_THREADS = 256, FEW_WARPS = 8;
constexpr uint32_t FEW_MAX_R = 256;      // pairs (one thread each in the prologues)
constexpr uint32_t FEW_MAX_TOKENS = 64;  // rows of mlp_down's per-warp sums
constexpr uint32_t TILES = 2;            // tiles of 16 rows a warp works on at once
constexpr uint32_t UP_PARTS = 4;         // mlp_up: warps that share a pair of tiles, each a part of hidden
constexpr uint32_t RING = 4;             // steps of a warp in flight
constexpr size_t UP_RING = FEW_WARPS * RING * TILES * 1024;
constexpr size_t FEW_SMEM = 220 * 1024;

// Planes of x by its type, of h by the result's.
constexpr int x_planes(int dt) { return dt == DT_F32 ? 2 : 1; }
__host__ __device__ constexpr int h_planes(int out_dtype) { return out_dtype == DT_BF16 ? 1 : 2; }

// One step of one pair's x or h, 128 values: planes [plane][unit 4][64 bytes], then
// (factor, sum of the values) of each unit, f32.
__host__ __device__ constexpr uint32_t step_bytes(int planes) { return (uint32_t)planes * 256u + 32u; }

// --------------------------------------------------------------------- codes

// Eight 4-bit codes of a word as f16 pairs: affine (0, 4), (1, 5), (2, 6), (3, 7) times
// 2^-24, the second and fourth pair 16 times that; E2M1 (0, 1), (2, 3), (4, 5), (6, 7).
template <int KIND>
__device__ __forceinline__ void expand(uint32_t w, uint32_t (&p)[4]) {
    if constexpr (KIND == K_AFF4) {
        p[0] = w & 0x000F000Fu;
        p[1] = w & 0x00F000F0u;
        p[2] = (w >> 8) & 0x000F000Fu;
        p[3] = (w >> 8) & 0x00F000F0u;
    } else {
        asm("{.reg .b8 a, b, c, d; mov.b32 {a, b, c, d}, %4; cvt.rn.f16x2.e2m1x2 %0, a; cvt.rn.f16x2.e2m1x2 %1, b; "
            "cvt.rn.f16x2.e2m1x2 %2, c; cvt.rn.f16x2.e2m1x2 %3, d;}"
            : "=r"(p[0]), "=r"(p[1]), "=r"(p[2]), "=r"(p[3])
            : "r"(w));
    }
}
// What expand()'s values have to be multiplied by.
template <int KIND> constexpr float code_unit = KIND == K_AFF4 ? 16777216.f : 1.f;
template <int KIND> constexpr bool affine_kind = KIND == K_AFF4;

// Place of value c of a unit among its 32 f16 values, as expand() pairs the codes, and
// whether it meets a code of the 16-fold pairs.
__device__ __forceinline__ uint32_t b_place(bool affine, uint32_t c) {
    return affine ? (c & ~7u) + 2u * (c & 3u) + ((c >> 2) & 1u) : c;
}
__device__ __forceinline__ bool b_sixteenth(bool affine, uint32_t c) { return affine && (c & 1u); }

__device__ __forceinline__ void mma(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                    uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t to_f16x2(float lo, float hi) {
    uint32_t d;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
    return d;
}
// Two E4M3 bytes.
__device__ __forceinline__ void from_e4m3x2(uint32_t v, float &a, float &b) {
    uint32_t f;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(f) : "h"((uint16_t)v));
    a = f16_bits_to_f32(f & 0xFFFFu);
    b = f16_bits_to_f32(f >> 16);
}

// Power of two that brings a unit whose largest |value| has these bits into [2^14, 2^15)
// (less for values below 2^-112), and its inverse.
__device__ __forceinline__ void unit_scale(uint32_t maxbits, float &scale, float &factor) {
    const uint32_t e = max(maxbits >> 23, 15u);
    scale = __uint_as_float((268u - e) << 23);
    factor = __uint_as_float((e - 14u) << 23);
}

// Bytes of one row's scales.
__host__ __device__ inline uint32_t scale_bytes(int kind, uint32_t groups) {
    return kind == K_AFF4 ? groups * 2u : groups;
}

// ------------------------------------------------------------------ one step

// What a lane needs of one step beside the weights: B registers of each block of
// columns, and for the two units of its accumulator columns the factors and, affine, the
// sums of x.
template <int NB>
struct StepB {
    uint32_t b[NB][16];
    float f[NB][2], xs[NB][2];
};

// From the pairs' step images at `base`, `stride` bytes apart; pairs at and past np are
// 0, as are the lanes whose k are not their column's unit: they read `zeros` (64 bytes).
template <int KIND, int PLANES, int NB>
__device__ __forceinline__ void load_step(StepB<NB> &S, const uint8_t *base, uint32_t stride, const uint8_t *zeros,
                                          uint32_t np, uint32_t lane) {
    const uint32_t q = lane & 3u;
    const bool active = ((lane >> 2) & 3u) == q;  // this lane's k of column lane / 4 are that column's unit
#pragma unroll
    for (uint32_t n = 0; n < NB; n++) {
        const uint32_t set = 2u * n + (lane >> 4), pair = set / PLANES, plane = set % PLANES;
        uint32_t(&b)[16] = S.b[n];
        const uint4 *v = (const uint4 *)(active && pair < np ? base + pair * stride + plane * 256u + q * 64u : zeros);
#pragma unroll
        for (int i = 0; i < 4; i++) {
            const uint4 x = v[i];
            b[4 * i] = x.x; b[4 * i + 1] = x.y; b[4 * i + 2] = x.z; b[4 * i + 3] = x.w;
        }
        // the lane's accumulator columns 2q, 2q + 1: units 2 (q mod 2) and the next of set 2n + q / 2
        const uint32_t cset = 2u * n + (q >> 1), cpair = cset / PLANES, cplane = cset % PLANES;
        const float4 f = *(const float4 *)(cpair < np ? base + cpair * stride + PLANES * 256u + (q & 1u) * 16u : zeros);
        const float unit = cplane ? code_unit<KIND> * 4.8828125e-4f : code_unit<KIND>;  // 2^-11
        S.f[n][0] = f.x * unit;
        S.f[n][1] = f.z * unit;
        S.xs[n][0] = cplane ? 0.f : f.y;  // the bias once a pair
        S.xs[n][1] = cplane ? 0.f : f.w;
    }
}

// Scales (and affine biases) that a lane applies: of rows r and r + 8 and the two units of
// its accumulator columns; NVFP4 units have two.
template <int KIND>
struct Scales {
    static constexpr int PARTS = KIND == K_NVFP4 ? 2 : 1;
    float s[PARTS][4];  // (row r, unit 0), (r, 1), (r + 8, 0), (r + 8, 1)
    float b[4];
};

// From the two rows' scales and biases, at the units' entries i0, i1 (affine: of their
// groups; one group for both where `same`).
template <int KIND>
__device__ __forceinline__ void load_scales(Scales<KIND> &S, const uint8_t *sa, const uint8_t *sb, const uint8_t *ba,
                                            const uint8_t *bb, uint32_t i0, uint32_t i1, bool same) {
    if constexpr (KIND == K_AFF4) {
        S.s[0][0] = S.s[0][1] = bf16_bits_to_f32(((const unsigned short *)sa)[i0]);
        S.s[0][2] = S.s[0][3] = bf16_bits_to_f32(((const unsigned short *)sb)[i0]);
        S.b[0] = S.b[1] = bf16_bits_to_f32(((const unsigned short *)ba)[i0]);
        S.b[2] = S.b[3] = bf16_bits_to_f32(((const unsigned short *)bb)[i0]);
        if (!same) {
            S.s[0][1] = bf16_bits_to_f32(((const unsigned short *)sa)[i1]);
            S.s[0][3] = bf16_bits_to_f32(((const unsigned short *)sb)[i1]);
            S.b[1] = bf16_bits_to_f32(((const unsigned short *)ba)[i1]);
            S.b[3] = bf16_bits_to_f32(((const unsigned short *)bb)[i1]);
        }
    } else if constexpr (KIND == K_MXFP4) {
        S.s[0][0] = e8m0_to_f32(sa[i0]);
        S.s[0][1] = e8m0_to_f32(sa[i1]);
        S.s[0][2] = e8m0_to_f32(sb[i0]);
        S.s[0][3] = e8m0_to_f32(sb[i1]);
    } else {
        constexpr int L = Scales<KIND>::PARTS - 1;
        from_e4m3x2(((const unsigned short *)sa)[i0], S.s[0][0], S.s[L][0]);
        from_e4m3x2(((const unsigned short *)sa)[i1], S.s[0][1], S.s[L][1]);
        from_e4m3x2(((const unsigned short *)sb)[i0], S.s[0][2], S.s[L][2]);
        from_e4m3x2(((const unsigned short *)sb)[i1], S.s[0][3], S.s[L][3]);
    }
}

// 16 rows x 4 units: wa, wb the lane's unit of rows r and r + 8.
template <int KIND, int NB>
__device__ __forceinline__ void tile_step(const uint4 wa, const uint4 wb, const StepB<NB> &S, const Scales<KIND> &C,
                                          float (&acc)[NB][2]) {
    const uint32_t a[4] = {wa.x, wa.y, wa.z, wa.w}, b[4] = {wb.x, wb.y, wb.z, wb.w};
    constexpr int PARTS = Scales<KIND>::PARTS, WPP = 4 / PARTS;  // words a part
#pragma unroll
    for (int h = 0; h < PARTS; h++) {
        float c[NB][4];
#pragma unroll
        for (int n = 0; n < NB; n++) c[n][0] = c[n][1] = c[n][2] = c[n][3] = 0.f;
#pragma unroll
        for (int i = 0; i < WPP; i++) {
            const int w = h * WPP + i;
            uint32_t pa[4], pb[4];
            expand<KIND>(a[w], pa);
            expand<KIND>(b[w], pb);
#pragma unroll
            for (int n = 0; n < NB; n++) {
                mma(c[n], pa[0], pb[0], pa[1], pb[1], S.b[n][4 * w], S.b[n][4 * w + 1]);
                mma(c[n], pa[2], pb[2], pa[3], pb[3], S.b[n][4 * w + 2], S.b[n][4 * w + 3]);
            }
        }
#pragma unroll
        for (int n = 0; n < NB; n++) {
            acc[n][0] = fmaf(C.s[h][0], c[n][0] * S.f[n][0], fmaf(C.s[h][1], c[n][1] * S.f[n][1], acc[n][0]));
            acc[n][1] = fmaf(C.s[h][2], c[n][2] * S.f[n][0], fmaf(C.s[h][3], c[n][3] * S.f[n][1], acc[n][1]));
        }
    }
    if constexpr (affine_kind<KIND>) {
#pragma unroll
        for (int n = 0; n < NB; n++) {
            acc[n][0] = fmaf(C.b[0], S.xs[n][0], fmaf(C.b[1], S.xs[n][1], acc[n][0]));
            acc[n][1] = fmaf(C.b[2], S.xs[n][0], fmaf(C.b[3], S.xs[n][1], acc[n][1]));
        }
    }
}

// ------------------------------------------------------------------- routing

// The distinct valid experts of at most 256 pairs as bits, ascending ranks by prefix
// counts. All threads of the CTA call it; shared arrays of 32 and 33.
__device__ __forceinline__ uint32_t expert_mask(uint32_t id, bool valid, uint32_t *mask, uint32_t *base) {
    const uint32_t tid = threadIdx.x;
    if (tid < 32) mask[tid] = 0u;
    __syncthreads();
    if (valid) atomicOr(&mask[id >> 5], 1u << (id & 31u));
    __syncthreads();
    if (tid < 32) {
        uint32_t n = __popc(mask[tid]), before = n;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const uint32_t o = __shfl_up_sync(FULL, before, d);
            if (tid >= (uint32_t)d) before += o;
        }
        base[tid] = before - n;
        if (tid == 31) base[32] = before;
    }
    __syncthreads();
    return base[32];
}

template <int N>
__device__ __forceinline__ void wait_groups() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// Thread block clusters: this block's rank, the barrier, and a load from the shared
// memory of the block of another rank at this block's address.
__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ float cluster_load(uint32_t addr, uint32_t rank) {
    float v;
    asm volatile("{.reg .u32 a; mapa.shared::cluster.u32 a, %1, %2; ld.shared::cluster.f32 %0, [a];}"
                 : "=f"(v)
                 : "r"(addr), "r"(rank)
                 : "memory");
    return v;
}

// --------------------------------------------------------------- projections

struct FewParams {
    const void *x;
    const uint32_t *ids;
    const float *weights;
    const uint8_t *w1, *w2;          // packed codes, gate_up and down
    const uint8_t *s1, *s2;          // scales
    const uint8_t *a1, *a2;          // affine biases, or scale2
    const void *bias1, *bias2;       // expert biases, or null
    const void *residual;
    void *out;
    uint8_t *hf;                     // h: [R][steps of inter][step_bytes(planes of h)]
    uint32_t *err;
    uint32_t m, R, S, E, H, I;       // H hidden, I inter
    uint32_t g1, g2, gshift1, gshift2;  // groups of a row; log2(units of 32 a group)
    int x_dtype, out_dtype, bias1_dtype, bias2_dtype, act;
    int scale2_kind, down_affine;    // 1: the down projection is NVFP4 (scale2 in a2); affine
    uint32_t cluster;                // mlp_down: blocks that share 32 columns
};

// Four consecutive x values.
template <int XT>
__device__ __forceinline__ float4 load_x4(const void *x, size_t i) {
    if constexpr (XT == DT_F32) {
        return __ldg((const float4 *)((const float *)x + i));
    } else {
        const uint2 v = __ldg((const uint2 *)((const uint16_t *)x + i));
        if constexpr (XT == DT_BF16)
            return make_float4(__uint_as_float(v.x << 16), __uint_as_float(v.x & 0xFFFF0000u),
                               __uint_as_float(v.y << 16), __uint_as_float(v.y & 0xFFFF0000u));
        else
            return make_float4(f16_bits_to_f32(v.x & 0xFFFFu), f16_bits_to_f32(v.x >> 16),
                               f16_bits_to_f32(v.y & 0xFFFFu), f16_bits_to_f32(v.y >> 16));
    }
}

// A warp writes one step image: lane l holds values 4l .. 4l+3 (unit l / 8).
template <int KIND, int PLANES>
__device__ __forceinline__ void write_step(uint8_t *dst, float4 v, uint32_t lane) {
    const uint32_t M = 0x7FFFFFFFu;
    uint32_t mb = max(max(__float_as_uint(v.x) & M, __float_as_uint(v.y) & M),
                      max(__float_as_uint(v.z) & M, __float_as_uint(v.w) & M));
    float sum = (v.x + v.y) + (v.z + v.w);
#pragma unroll
    for (int d = 1; d < 8; d <<= 1) {
        mb = max(mb, __shfl_xor_sync(FULL, mb, d));
        if constexpr (affine_kind<KIND>) sum += __shfl_xor_sync(FULL, sum, d);
    }
    float scale, factor;
    unit_scale(mb, scale, factor);
    if constexpr (affine_kind<KIND>) {
        // a word's pairs are (0, 4), (1, 5) for the even lane and (2, 6), (3, 7) for the odd one
        const bool odd = lane & 1u;
        const float s0 = odd ? v.x : v.z, s1 = odd ? v.y : v.w;
        const float r0 = __shfl_xor_sync(FULL, s0, 1), r1 = __shfl_xor_sync(FULL, s1, 1);
        const float sixteenth = scale * 0.0625f;
        v = odd ? make_float4(r0 * scale, v.z * scale, r1 * sixteenth, v.w * sixteenth)
                : make_float4(v.x * scale, r0 * scale, v.y * sixteenth, r1 * sixteenth);
    } else {
        v = make_float4(v.x * scale, v.y * scale, v.z * scale, v.w * scale);
    }
    uint2 *p = (uint2 *)(dst + lane * 8u);
#pragma unroll
    for (int k = 0; k < PLANES; k++, p += 32) {
        const uint2 o = make_uint2(to_f16x2(v.x, v.y), to_f16x2(v.z, v.w));
        *p = o;
        if (k + 1 < PLANES) {
            v.x = (v.x - f16_bits_to_f32(o.x & 0xFFFFu)) * 2048.f;
            v.y = (v.y - f16_bits_to_f32(o.x >> 16)) * 2048.f;
            v.z = (v.z - f16_bits_to_f32(o.y & 0xFFFFu)) * 2048.f;
            v.w = (v.w - f16_bits_to_f32(o.y >> 16)) * 2048.f;
        }
    }
    if ((lane & 7u) == 0u) *(float2 *)(dst + PLANES * 256 + (lane >> 3) * 8u) = make_float2(factor, sum);
}

// mlp_up. grid (inter / 32, ranks of distinct experts). A CTA holds 32 columns of h, a
// unit of mlp_down (64 weight rows: tile t pairs gate rows 8t..8t+7 with up rows
// 8t..8t+7, so that a lane's two accumulator rows are the gate and the up of one
// column). Each pair of tiles has four warps, which take the steps of 128 codes in
// turn; x is written as step images once for all of them. Two tiles a warp share a
// step's B registers and its loop.
template <int KIND, int XT, int NB>
__global__ void __launch_bounds__(FEW_THREADS, NB <= 2 ? 2 : 1) mlp_up(const FewParams P) {
    constexpr int PLANES = x_planes(XT), PP = 2 * NB / PLANES;  // pairs a pass
    constexpr uint32_t STAGE = TILES * 2 * 512, XSTEP = step_bytes(PLANES);
    extern __shared__ __align__(16) uint8_t sm[];
    __shared__ __align__(16) uint8_t zeros[64];
    __shared__ uint32_t mask[32], base[33], wcount[FEW_WARPS], pairs[FEW_MAX_R], expert_s;

    const uint32_t tid = threadIdx.x, warp = tid >> 5, lane = tid & 31u;
    if (tid < 16) ((uint32_t *)zeros)[tid] = 0u;
    // mlp_down may start from here on: what came before this kernel is complete
    ptx::griddep_wait();
    ptx::griddep_launch_dependents();

    // the expert of this rank and its pairs, ascending
    uint32_t e, np;
    if (P.R <= 32u) {  // each warp by itself; ranks in the order of the experts' first pairs
        const uint32_t id = lane < P.R ? __ldg(P.ids + lane) : FULL;
        const bool valid = id < P.E;
        if (blockIdx.x == 0 && blockIdx.y == 0 && warp == 0 && lane < P.R && !valid) atomicOr(P.err, ERR_BAD_ID);
        const uint32_t same = __match_any_sync(FULL, id);
        uint32_t firsts = __ballot_sync(FULL, valid && __ffs(same) - 1u == lane);
        if (blockIdx.y >= __popc(firsts)) return;
        for (uint32_t i = 0; i < blockIdx.y; i++) firsts &= firsts - 1u;
        e = __shfl_sync(FULL, id, __ffs(firsts) - 1);
        const uint32_t mine = __ballot_sync(FULL, valid && id == e);
        np = __popc(mine);
        if (warp == 0 && valid && id == e) pairs[__popc(mine & ((1u << lane) - 1u))] = lane;
    } else {
        const uint32_t id = tid < P.R ? __ldg(P.ids + tid) : FULL;
        const bool valid = id < P.E;
        if (blockIdx.x == 0 && blockIdx.y == 0 && tid < P.R && !valid) atomicOr(P.err, ERR_BAD_ID);
        if (blockIdx.y >= expert_mask(id, valid, mask, base)) return;
        if (tid < 32 && base[tid] <= blockIdx.y && blockIdx.y < base[tid + 1]) {
            uint32_t m = mask[tid];
            for (uint32_t i = base[tid]; i < blockIdx.y; i++) m &= m - 1u;
            expert_s = tid * 32u + __ffs(m) - 1u;
        }
        __syncthreads();
        e = expert_s;
        const uint32_t mine = __ballot_sync(FULL, valid && id == e);
        if (lane == 0) wcount[warp] = __popc(mine);
        __syncthreads();
        uint32_t at = 0;
        np = 0;
#pragma unroll
        for (uint32_t i = 0; i < FEW_WARPS; i++) {
            if (i < warp) at += wcount[i];
            np += wcount[i];
        }
        if (valid && id == e) pairs[at + __popc(mine & ((1u << lane) - 1u))] = tid;
    }

    const uint32_t r = lane >> 2, q = lane & 3u, tp = warp & 1u, part = warp >> 1;
    const uint32_t nu = P.H / 32u, steps = (nu + 3u) / 4u;
    const uint32_t row_bytes = P.H / 2u;
    const uint32_t c0 = blockIdx.x * 32u;
    const uint32_t srow = scale_bytes(KIND, P.g1);
    uint8_t *const images = sm + FEW_WARPS * RING * STAGE;  // [pair][step]
    uint8_t *const s_s = images + PP * steps * XSTEP;
    uint8_t *const b_s = s_s + 64u * srow;
    const uint32_t sm0 = ptx::smem_u32(sm);
    const uint32_t ring = sm0 + warp * RING * STAGE + lane * 16u;
    // this lane's unit of its rows of the first tile
    const uint8_t *const wrow = P.w1 + ((size_t)e * 2u * P.I + c0 + 16u * tp + r) * row_bytes + q * 16u;
    const size_t up = (size_t)P.I * row_bytes, next = 8u * (size_t)row_bytes;

    const uint8_t *src = wrow;
    uint32_t ju = 0, is = 0;  // next step to request, its slot
    auto issue = [&]() {
        if (ju < steps) {
            const uint32_t size = 4u * ju + q < nu ? 16u : 0u;  // past the row nothing is read, zeros are stored
            const uint8_t *g = size ? src : wrow;
            ptx::cp_async_16(ring + is, g, size);
            ptx::cp_async_16(ring + is + 512u, g + up, size);
            g += next;
            ptx::cp_async_16(ring + is + 1024u, g, size);
            ptx::cp_async_16(ring + is + 1536u, g + up, size);
            src += UP_PARTS * 64u;
            is = (is + STAGE) & (RING * STAGE - 1u);
            ju += UP_PARTS;
        }
        ptx::cp_async_commit();
    };
    auto restart = [&]() {
        src = wrow + part * 64u;
        ju = part;
        is = 0u;
#pragma unroll
        for (uint32_t i = 0; i < RING; i++) issue();
    };

    // scales (and affine biases) of the 64 rows: two blocks of 32 contiguous rows each
    for (uint32_t o = tid * 16u; o < 64u * srow; o += FEW_THREADS * 16u) {
        const uint32_t half = o >= 32u * srow;
        const size_t so = ((size_t)e * 2u * P.I + half * P.I + c0) * srow + (o - half * 32u * srow);
        ptx::cp_async_16(sm0 + (uint32_t)(s_s - sm) + o, P.s1 + so, 16);
        if constexpr (affine_kind<KIND>) ptx::cp_async_16(sm0 + (uint32_t)(b_s - sm) + o, P.a1 + so, 16);
    }
    ptx::cp_async_commit();
    restart();
    __syncthreads();  // pairs[]

    for (uint32_t pb = 0; pb < np; pb += PP) {
        const uint32_t npass = tmin<uint32_t>(PP, np - pb);
        if (pb) restart();
        for (uint32_t p = 0; p < npass; p++) {
            const size_t xrow = (size_t)(pairs[pb + p] / P.S) * P.H + 4u * lane;
#pragma unroll 4
            for (uint32_t j = warp; j < steps; j += FEW_WARPS) {
                const float4 v = j * 128u + 4u * lane < P.H ? load_x4<XT>(P.x, xrow + j * 128u)
                                                            : make_float4(0.f, 0.f, 0.f, 0.f);
                write_step<KIND, PLANES>(images + (p * steps + j) * XSTEP, v, lane);
            }
        }
        // what the epilogue of this warp's pair needs, requested now (a pass has at most 8)
        const bool mine = warp < npass;
        const uint32_t p_e = mine ? pairs[pb + warp] : 0u, c = c0 + lane;
        float weight = 0.f, bg = 0.f, bu = 0.f;
        if (mine) {
            weight = __ldg(P.weights + p_e);
            if (P.scale2_kind) weight *= __ldg((const float *)P.a2 + e);
            bg = load_bias(P.bias1, P.bias1_dtype, (size_t)e * 2u * P.I + c);
            bu = load_bias(P.bias1, P.bias1_dtype, (size_t)e * 2u * P.I + P.I + c);
        }
        if (pb == 0) wait_groups<RING>();  // the scales' group is the oldest
        __syncthreads();                   // images, and the other threads' parts of the scales

        float acc[TILES][NB][2];
#pragma unroll
        for (uint32_t t = 0; t < TILES; t++)
#pragma unroll
            for (int n = 0; n < NB; n++) acc[t][n][0] = acc[t][n][1] = 0.f;
        const uint8_t *st = sm + warp * RING * STAGE + lane * 16u;
        const uint8_t *const sr = s_s + (16u * tp + r) * srow, *const br = b_s + (16u * tp + r) * srow;
        const uint8_t *img = images + part * XSTEP;
        uint32_t slot = 0;
        for (uint32_t j = part; j < steps; j += UP_PARTS) {
            StepB<NB> B;
            load_step<KIND, PLANES, NB>(B, img, steps * XSTEP, zeros, npass, lane);
            img += UP_PARTS * XSTEP;
            const uint32_t u = 4u * j + 2u * (q & 1u);
            uint32_t i0 = tmin<uint32_t>(u, nu - 1u), i1 = tmin<uint32_t>(u + 1u, nu - 1u);
            if constexpr (affine_kind<KIND>) {
                i0 >>= P.gshift1;
                i1 >>= P.gshift1;
            }
            wait_groups<RING - 1>();
#pragma unroll
            for (uint32_t t = 0; t < TILES; t++) {
                const uint4 wa = *(const uint4 *)(st + slot + t * 1024u), wb = *(const uint4 *)(st + slot + t * 1024u + 512u);
                Scales<KIND> C;
                const uint32_t o = t * 8u * srow, ou = o + 32u * srow;
                load_scales<KIND>(C, sr + o, sr + ou, br + o, br + ou, i0, i1, P.gshift1 != 0u);
                tile_step<KIND, NB>(wa, wb, B, C, acc[t]);
            }
            slot = (slot + STAGE) & (RING * STAGE - 1u);
            issue();
        }
        asm volatile("cp.async.wait_all;" ::: "memory");
        __syncthreads();  // the ring is free: the warps' sums go there
        float *const red = (float *)sm;  // [part][pair][gate / up][32 columns]
#pragma unroll
        for (uint32_t t = 0; t < TILES; t++)
#pragma unroll
            for (int n = 0; n < NB; n++)
#pragma unroll
                for (int h = 0; h < 2; h++) {
                    float v = acc[t][n][h];
                    v += __shfl_xor_sync(FULL, v, 1);
                    if constexpr (PLANES == 2) v += __shfl_xor_sync(FULL, v, 2);
                    if (PLANES == 2 ? q == 0u : !(q & 1u)) {
                        const uint32_t p = PLANES == 2 ? n : 2u * n + (q >> 1);
                        red[((part * PP + p) * 2u + h) * 32u + 16u * tp + 8u * t + r] = v;
                    }
                }
        __syncthreads();
        if (mine) {  // one warp a pair: lane = column of h
            float g = 0.f, v = 0.f;
#pragma unroll
            for (uint32_t k = 0; k < UP_PARTS; k++) {
                g += red[((k * PP + warp) * 2u) * 32u + lane];
                v += red[((k * PP + warp) * 2u + 1u) * 32u + lane];
            }
            if constexpr (KIND == K_NVFP4) {
                const float s2 = __ldg((const float *)P.a1 + e);
                g *= s2;
                v *= s2;
            }
            float h = glu_act(P.act, g + bg) * (v + bu) * weight;
            // this unit of the pair's step image
            const int planes = h_planes(P.out_dtype);
            const uint32_t iu = P.I / 32u, un = blockIdx.x & 3u;
            uint8_t *img_h = P.hf + ((size_t)p_e * ((iu + 3u) / 4u) + (blockIdx.x >> 2)) * step_bytes(planes);
            float sum = h;
#pragma unroll
            for (int d = 16; d > 0; d >>= 1) sum += __shfl_xor_sync(FULL, sum, d);
            float scale, factor;
            unit_scale(__reduce_max_sync(FULL, __float_as_uint(h) & 0x7FFFFFFFu), scale, factor);
            h *= scale;
            if (b_sixteenth(P.down_affine, lane)) h *= 0.0625f;
            uint16_t *dst = (uint16_t *)(img_h + un * 64u) + b_place(P.down_affine, lane);
            for (int k = 0; k < planes; k++, dst += 128) {
                const __half b = __float2half_rn(h);
                *dst = __half_as_ushort(b);
                h = (h - __half2float(b)) * 2048.f;
            }
            float2 *fs = (float2 *)(img_h + planes * 256);
            if (lane == 0) fs[un] = make_float2(factor, sum);
            // units past inter in the last step are zero
            if (blockIdx.x + 1u == iu)
                for (uint32_t z = un + 1u; z < 4u; z++) {
                    for (int k = 0; k < planes; k++) ((uint16_t *)(img_h + k * 256 + z * 64u))[lane] = 0;
                    if (lane == 0) fs[z] = make_float2(0.f, 0.f);
                }
        }
        if (pb + PP < np) __syncthreads();  // red is read before the next pass's copies land there
    }
}

// Scales of one step and row in mlp_down's ring: whole aligned words around the bytes.
constexpr uint32_t DN_SROW = 12;

// mlp_down. grid (hidden / 32 * cluster), a cluster of blocks for 32 columns of out (two
// tiles a warp). The cluster's warps share the work items, (expert, part of its steps);
// each keeps sums of its own for every token, added in warp order within a block and in
// rank order through distributed shared memory: no atomics, one order. Weights and
// scales do not depend on mlp_up, so the ring's first steps are requested before
// waiting for it.
template <int KIND, int NPL, int NB>
__global__ void __launch_bounds__(FEW_THREADS, NB <= 2 ? 2 : 1) mlp_down(const FewParams P) {
    constexpr uint32_t PP = 2 * NB / NPL;  // pairs a pass
    constexpr uint32_t HSTEP = step_bytes(NPL), WBYTES = TILES * 2 * 512, SBYTES = 32 * DN_SROW;
    constexpr uint32_t STAGE = WBYTES + PP * HSTEP + SBYTES * (affine_kind<KIND> ? 2 : 1);
    extern __shared__ __align__(16) uint8_t sm[];
    __shared__ __align__(16) uint8_t zeros[64];
    __shared__ uint32_t mask[32], base[33], ids_s[FEW_MAX_R], first[FEW_MAX_R + 1], pairs[FEW_MAX_R],
        experts[FEW_MAX_R];

    const uint32_t tid = threadIdx.x, warp = tid >> 5, lane = tid & 31u;
    if (tid < 16) ((uint32_t *)zeros)[tid] = 0u;
    const uint32_t id = tid < P.R ? __ldg(P.ids + tid) : FULL;  // complete before mlp_up began
    const bool valid = id < P.E;
    ids_s[tid] = valid ? id : FULL;
    first[tid] = 0u;
    if (tid == 0) first[FEW_MAX_R] = 0u;
    const uint32_t D = expert_mask(id, valid, mask, base);
    // pairs by expert: rank, count, first, place (stable)
    uint32_t rank = 0, place = 0;
    if (valid) {
        rank = base[id >> 5] + __popc(mask[id >> 5] & ((1u << (id & 31u)) - 1u));
        atomicAdd(&first[rank + 1u], 1u);
        experts[rank] = id;
        for (uint32_t t = 0; t < tid; t++) place += ids_s[t] == id;
    }
    float *const ysm = (float *)(sm + FEW_WARPS * RING * STAGE);  // [warp][token][32]
    for (uint32_t o = tid; o < FEW_WARPS * P.m * 32u; o += FEW_THREADS) ysm[o] = 0.f;
    __syncthreads();
    if (warp == 0) {
        uint32_t carry = 0;
        for (uint32_t o = 0; o < D; o += 32) {
            uint32_t v = o + lane < D ? first[o + lane + 1u] : 0u;
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
                const uint32_t y = __shfl_up_sync(FULL, v, d);
                if (lane >= (uint32_t)d) v += y;
            }
            v += carry;
            if (o + lane < D) first[o + lane + 1u] = v;
            carry = __shfl_sync(FULL, v, 31);
        }
    }
    __syncthreads();
    if (valid) pairs[first[rank] + place] = tid;
    __syncthreads();

    const uint32_t r = lane >> 2, q = lane & 3u;
    const uint32_t nu = P.I / 32u, steps = (nu + 3u) / 4u, row_bytes = P.I / 2u;
    const uint32_t crank = P.cluster > 1u ? cluster_rank() : 0u, warps = P.cluster * FEW_WARPS;
    const uint32_t row0 = blockIdx.x / P.cluster * 32u;
    const uint32_t srow = scale_bytes(KIND, P.g2);
    // about four items a warp
    const uint32_t parts = D ? tmin<uint32_t>((4u * warps + D - 1u) / D, steps) : 1u;
    const uint32_t items = D * parts;
    uint8_t *const wsm = sm + warp * RING * STAGE;
    const uint32_t ring = ptx::smem_u32(wsm);

    // a position in the warp's list of steps: item, its first step, step, first pair of
    // the pass and of the expert, pairs of the expert
    struct Pos {
        uint32_t item, x, j0, j, pb, first, cnt;
    };
    auto enter = [&](Pos &p) {
        if (p.item < items) {
            p.x = p.item / parts;
            p.j = p.j0 = p.item - p.x * parts;
            p.pb = 0u;
            p.first = first[p.x];
            p.cnt = first[p.x + 1u] - p.first;
        }
    };
    auto advance = [&](Pos &p) {  // whether a pass ended
        p.j += parts;
        if (p.j < steps) return false;
        p.j = p.j0;
        p.pb += PP;
        if (p.pb >= p.cnt) {
            p.item += warps;
            enter(p);
        }
        return true;
    };
    // requests: the weights and their scales, then h
    const uint8_t *w0 = nullptr, *s0 = nullptr, *b0 = nullptr;
    auto start_w = [&](const Pos &p) {
        if (p.item >= items) return;
        const size_t row = (size_t)experts[p.x] * P.H + row0;
        w0 = P.w2 + (row + r) * row_bytes + q * 16u;          // the lane's unit of row r, step 0
        s0 = P.s2 + (row + lane) * srow;                      // scales: lane = row
        if constexpr (affine_kind<KIND>) b0 = P.a2 + (row + lane) * srow;
    };
    // bytes of a step's scales in their row
    const uint32_t sfirst = affine_kind<KIND> ? 0u : KIND == K_NVFP4 ? 8u : 4u;
    auto scale_at = [&](uint32_t j) { return affine_kind<KIND> ? ((4u * j) >> P.gshift2) * 2u : sfirst * j; };
    auto issue_w = [&](const Pos &p, uint32_t stage) {
        const uint32_t size = 4u * p.j + q < nu ? 16u : 0u;
        const uint8_t *src = w0 + (size ? p.j * 64u : 0u);
        const uint32_t st = ring + stage + lane * 16u;
#pragma unroll
        for (uint32_t t = 0; t < 2 * TILES; t++) ptx::cp_async_16(st + t * 512u, src + t * 8u * row_bytes, size);
        // the aligned words that hold bytes [o, end) of this lane's row
        const uint32_t o = scale_at(p.j), end = tmin<uint32_t>(scale_at(p.j + 1u) + (P.gshift2 > 2u ? 2u : 0u), srow);
        const uint32_t ss = ring + stage + WBYTES + PP * HSTEP + lane * DN_SROW;
        const uint32_t off = (uint32_t)((uintptr_t)(s0 + o) & 3u);
#pragma unroll
        for (uint32_t k = 0; k < 3; k++)
            if (o + 4u * k < end + off) {
                ptx::cp_async_4(ss + 4u * k, s0 + o - off + 4u * k, 4);
                if constexpr (affine_kind<KIND>) ptx::cp_async_4(ss + SBYTES + 4u * k, b0 + o - off + 4u * k, 4);
            }
    };
    uint32_t ho[PP];  // the pairs' offsets in hf
    auto start_h = [&](const Pos &p) {
        if (p.item >= items) return;
#pragma unroll
        for (uint32_t k = 0; k < PP; k++)
            ho[k] = p.pb + k < p.cnt ? pairs[p.first + p.pb + k] * steps * HSTEP + lane * 16u : 0u;
    };
    auto issue_h = [&](const Pos &p, uint32_t stage) {
        const uint32_t st = ring + stage + WBYTES + lane * 16u;
        const uint8_t *src = P.hf + p.j * HSTEP;
#pragma unroll
        for (uint32_t k = 0; k < PP; k++)
            if (p.pb + k < p.cnt) {
#pragma unroll
                for (uint32_t o = 0; o < HSTEP; o += 512u)
                    if (lane * 16u + o < HSTEP) ptx::cp_async_16(st + k * HSTEP + o, src + ho[k] + o, 16);
            }
    };

    Pos ahead{crank * FEW_WARPS + warp, 0u, 0u, 0u, 0u, 0u, 0u};
    enter(ahead);
    Pos at = ahead;
    start_w(ahead);
    uint32_t issued = 0;
    for (; issued < RING && ahead.item < items; issued++) {
        issue_w(ahead, issued * STAGE);
        if (advance(ahead)) start_w(ahead);
    }
    ptx::cp_async_commit();
    ptx::griddep_wait();  // h
    Pos fill = at;
    start_h(fill);
    for (uint32_t i = 0; i < RING; i++) {
        if (i < issued) {
            issue_h(fill, i * STAGE);
            if (advance(fill)) start_h(fill);
        }
        ptx::cp_async_commit();
    }
    start_h(ahead);

    float acc[TILES][NB][2];
#pragma unroll
    for (uint32_t t = 0; t < TILES; t++)
#pragma unroll
        for (int n = 0; n < NB; n++) acc[t][n][0] = acc[t][n][1] = 0.f;
    uint32_t stage = 0;
    while (at.item < items) {
        wait_groups<RING - 1>();  // the oldest step: its weights came in an older group
        __syncwarp();             // and the other lanes' parts of the scales and of h
        const uint8_t *st = wsm + stage;
        StepB<NB> B;
        load_step<KIND, NPL, NB>(B, st + WBYTES, HSTEP, zeros, at.cnt - at.pb, lane);
        // entries of the step's scales, from its first one; past the row they are the last
        const uint32_t u = 2u * (q & 1u), last = nu - 1u - 4u * at.j;
        uint32_t i0 = tmin<uint32_t>(u, last), i1 = tmin<uint32_t>(u + 1u, last);
        if constexpr (affine_kind<KIND>) {
            const uint32_t g = (4u * at.j) >> P.gshift2;
            i0 = ((4u * at.j + i0) >> P.gshift2) - g;
            i1 = ((4u * at.j + i1) >> P.gshift2) - g;
        }
        const uint8_t *ss = st + WBYTES + PP * HSTEP;
        const uint32_t so = scale_at(at.j);
#pragma unroll
        for (uint32_t t = 0; t < TILES; t++) {
            // a row's bytes stand at their own address modulo 4 (arrays and row0 * srow are multiples of 16)
            const uint32_t ra = 16u * t + r, rb = ra + 8u;
            const uint8_t *sa = ss + ra * DN_SROW + ((ra * srow + so) & 3u), *sb = ss + rb * DN_SROW + ((rb * srow + so) & 3u);
            Scales<KIND> C;
            load_scales<KIND>(C, sa, sb, sa + SBYTES, sb + SBYTES, i0, i1, P.gshift2 != 0u);
            tile_step<KIND, NB>(*(const uint4 *)(st + t * 1024u + lane * 16u),
                                *(const uint4 *)(st + t * 1024u + 512u + lane * 16u), B, C, acc[t]);
        }
        const uint32_t pfirst = at.first + at.pb, pcnt = at.cnt - at.pb;
        const bool ended = advance(at);
        __syncwarp();  // every lane has read its stage
        if (ahead.item < items) {
            issue_w(ahead, stage);
            issue_h(ahead, stage);
            if (advance(ahead)) {
                start_w(ahead);
                start_h(ahead);
            }
        }
        ptx::cp_async_commit();
        stage = stage + STAGE == RING * STAGE ? 0u : stage + STAGE;
        if (ended) {  // end of a pass: into the tokens' sums
#pragma unroll
            for (uint32_t n = 0; n < NB; n++) {
                float v[TILES][2];
#pragma unroll
                for (uint32_t t = 0; t < TILES; t++)
#pragma unroll
                    for (int h = 0; h < 2; h++) {
                        v[t][h] = acc[t][n][h] + __shfl_xor_sync(FULL, acc[t][n][h], 1);
                        if constexpr (NPL == 2) v[t][h] += __shfl_xor_sync(FULL, v[t][h], 2);
                        acc[t][n][h] = 0.f;
                    }
                // one pair at a time: two of them may be one token's
#pragma unroll
                for (uint32_t k = 0; k < 2u / NPL; k++) {
                    const uint32_t p = n * (2u / NPL) + k;
                    if (q == 2u * k && p < pcnt) {
                        float *y = ysm + ((size_t)warp * P.m + pairs[pfirst + p] / P.S) * 32u + r;
#pragma unroll
                        for (uint32_t t = 0; t < TILES; t++) {
                            y[16u * t] += v[t][0];
                            y[16u * t + 8u] += v[t][1];
                        }
                    }
                    __syncwarp();
                }
            }
        }
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
    __syncthreads();
    float *const bsum = (float *)sm;  // this block's sums [token][32], where the ring was
    for (uint32_t o = tid; o < P.m * 32u; o += FEW_THREADS) {
        float y = 0.f;
#pragma unroll
        for (uint32_t w = 0; w < FEW_WARPS; w++) y += ysm[w * P.m * 32u + o];
        bsum[o] = y;
    }
    if (P.cluster > 1u) cluster_sync();
    else __syncthreads();
    const uint32_t baddr = ptx::smem_u32(bsum);
    for (uint32_t o = crank * FEW_THREADS + tid; o < P.m * 32u; o += P.cluster * FEW_THREADS) {
        const uint32_t t = o >> 5, c = row0 + (o & 31u);
        float y = bsum[o];
        if (P.cluster > 1u) {
            y = 0.f;
            for (uint32_t k = 0; k < P.cluster; k++) y += cluster_load(baddr + 4u * o, k);
        }
        if (P.bias2)
            for (uint32_t s = 0; s < P.S; s++) {
                const uint32_t e = ids_s[t * P.S + s];
                if (e != FULL)
                    y = fmaf(__ldg(P.weights + t * P.S + s), load_bias(P.bias2, P.bias2_dtype, (size_t)e * P.H + c), y);
            }
        const size_t oi = (size_t)t * P.H + c;
        if (P.residual) {
            // not through the read-only path: it may be out itself
            y += P.out_dtype == DT_F32 ? ((const float *)P.residual)[oi]
               : P.out_dtype == DT_BF16 ? __bfloat162float(((const __nv_bfloat16 *)P.residual)[oi])
                                        : __half2float(((const __half *)P.residual)[oi]);
        }
        store_out(P.out, P.out_dtype, oi, y);
    }
    if (P.cluster > 1u) cluster_sync();  // the other blocks have read this one's sums
}

// ------------------------------------------------------------------ launches

// mlp_up's shared memory beside the ring: the pass's step images and the rows' scales.
size_t up_fixed_bytes(int kind, uint32_t H, uint32_t groups, int x_dtype, uint32_t blocks) {
    const int planes = x_planes(x_dtype);
    return (size_t)(2u * blocks / planes) * ((H / 32u + 3u) / 4u) * step_bytes(planes) +
           64ull * scale_bytes(kind, groups) * (kind == K_AFF4 ? 2u : 1u);
}

template <int KIND, int XT, int NB>
cudaError_t up_t(const FewParams &P, cudaStream_t st) {
    const size_t smem = UP_RING + up_fixed_bytes(KIND, P.H, P.g1, XT, NB);
    auto kern = mlp_up<KIND, XT, NB>;
    static int smem_set[64];
    const cudaError_t e = ensure_dyn_smem(kern, smem, smem_set);
    if (e != cudaSuccess) return e;
    kern<<<dim3(P.I / 32u, tmin<uint32_t>(P.R, P.E)), FEW_THREADS, smem, st>>>(P);
    return cudaGetLastError();
}

constexpr size_t down_bytes(bool affine, int planes, int blocks) {
    return (size_t)FEW_WARPS * RING *
           (TILES * 1024 + (2 * blocks / planes) * step_bytes(planes) + 32 * DN_SROW * (affine ? 2 : 1));
}

template <int KIND, int NPL, int NB>
cudaError_t down_t(FewParams P, cudaStream_t st) {
    const size_t smem = down_bytes(affine_kind<KIND>, NPL, NB) + FEW_WARPS * 128ull * P.m;
    auto kern = mlp_down<KIND, NPL, NB>;
    static int smem_set[64];
    const cudaError_t e = ensure_dyn_smem(kern, smem, smem_set);
    if (e != cudaSuccess) return e;
    // blocks for two an SM or more, so that the SMs' shares are even
    P.cluster = 1u;
    while (P.cluster < 8u && P.H / 32u * P.cluster < 2u * 148u) P.cluster *= 2u;
    // a programmatic dependent of mlp_up: it requests its weights while mlp_up runs and
    // waits (griddepcontrol.wait) before it reads h
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(P.H / 32u * P.cluster);
    cfg.blockDim = dim3(FEW_THREADS);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = P.cluster;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, kern, P);
}

// Blocks of columns of a pass: room for 1 pair of an expert for a single token, else
// for the power of two above the mean when the pairs spread evenly, at least 2 and at
// most 8 planes (4 blocks); more pairs take further passes over the expert's rows.
uint32_t blocks_a_pass(const FewParams &P, uint32_t planes) {
    const uint32_t pairs = P.m == 1 ? 1u : P.R <= P.E ? 2u : P.R <= 2u * P.E ? 4u : 8u;
    return tmin<uint32_t>((pairs * planes + 1u) / 2u, 4u);
}

template <int KIND, int XT>
cudaError_t up_x(const FewParams &P, cudaStream_t st) {
    uint32_t blocks = blocks_a_pass(P, x_planes(XT));
    while (blocks > 1u && up_fixed_bytes(KIND, P.H, P.g1, XT, blocks) + UP_RING > FEW_SMEM) blocks /= 2u;
    switch (blocks) {
        case 1: return up_t<KIND, XT, 1>(P, st);
        case 2: return up_t<KIND, XT, 2>(P, st);
        default: return up_t<KIND, XT, 4>(P, st);
    }
}

template <int KIND>
cudaError_t up_k(const FewParams &P, cudaStream_t st) {
    if (P.x_dtype == DT_F32) return up_x<KIND, DT_F32>(P, st);
    if (P.x_dtype == DT_BF16) return up_x<KIND, DT_BF16>(P, st);
    return up_x<KIND, DT_F16>(P, st);
}

template <int KIND, int NPL>
cudaError_t down_p(const FewParams &P, cudaStream_t st) {
    uint32_t blocks = blocks_a_pass(P, NPL);
    while (blocks > 1u && down_bytes(affine_kind<KIND>, NPL, (int)blocks) + FEW_WARPS * 128ull * P.m > FEW_SMEM)
        blocks /= 2u;
    switch (blocks) {
        case 1: return down_t<KIND, NPL, 1>(P, st);
        case 2: return down_t<KIND, NPL, 2>(P, st);
        default: return down_t<KIND, NPL, 4>(P, st);
    }
}

template <int KIND>
cudaError_t down_k(const FewParams &P, cudaStream_t st) {
    return h_planes(P.out_dtype) == 1 ? down_p<KIND, 1>(P, st) : down_p<KIND, 2>(P, st);
}

bool projection_ok(const moe_expert_weights &w, uint32_t k) {
    const int kind = kind_of((int)w.fmt, (int)w.bits);
    if (kind != K_AFF4 && kind != K_NVFP4 && kind != K_MXFP4) return false;
    if (kind == K_AFF4) {
        const uint32_t u = w.group_size / 32u;  // units a group
        if (w.group_size % 32u != 0 || (u & (u - 1u)) != 0 || ((uintptr_t)w.aux & 15u)) return false;
    }
    if (kind == K_NVFP4 && ((uintptr_t)w.aux & 3u)) return false;
    return k % 32u == 0 && !(((uintptr_t)w.packed | (uintptr_t)w.scales) & 15u);
}

uint32_t log2_units(const moe_expert_weights &w) {
    uint32_t s = 0;
    while ((32u << s) < w.group_size) s++;
    return s;
}

}  // namespace

uint64_t mlp_few_workspace(uint32_t m, uint32_t inter, uint32_t S) {
    const uint64_t R = (uint64_t)m * S;
    return R <= FEW_MAX_R ? R * ((inter + 127ull) / 128ull) * step_bytes(h_planes(DT_F32)) : 0ull;
}

// Whole 32-code units of 16 aligned bytes and scale groups of whole units in both
// projections, at most 256 pairs of at most 64 tokens, x and the scales of a CTA's rows
// in shared memory beside the ring.
bool mlp_few_supported(const MlpArgs &a) {
    const uint64_t R = (uint64_t)a.m * a.S;
    if (R > FEW_MAX_R || a.m > FEW_MAX_TOKENS || a.E > MOE_ROUTE_MAX_EXPERTS) return false;
    if (!projection_ok(*a.gate_up, a.hidden) || !projection_ok(*a.down, a.inter)) return false;
    if ((uintptr_t)a.x & 15u) return false;
    const int k1 = kind_of((int)a.gate_up->fmt, (int)a.gate_up->bits);
    const int k2 = kind_of((int)a.down->fmt, (int)a.down->bits);
    // both with one block of columns
    const size_t up = UP_RING + up_fixed_bytes(k1, a.hidden, a.hidden / a.gate_up->group_size, a.x_dtype, 1);
    const size_t dn = down_bytes(k2 == K_AFF4, 1, 1) + FEW_WARPS * 128ull * a.m;
    return up <= FEW_SMEM && dn <= FEW_SMEM;
}

cudaError_t launch_mlp_few(const MlpArgs &a, uint32_t *err, void *hf, cudaStream_t st) {
    FewParams P{};
    P.x = a.x; P.ids = a.ids; P.weights = a.weights;
    P.w1 = (const uint8_t *)a.gate_up->packed; P.w2 = (const uint8_t *)a.down->packed;
    P.s1 = (const uint8_t *)a.gate_up->scales; P.s2 = (const uint8_t *)a.down->scales;
    P.a1 = (const uint8_t *)a.gate_up->aux; P.a2 = (const uint8_t *)a.down->aux;
    P.bias1 = a.gate_up->bias; P.bias2 = a.down->bias;
    P.bias1_dtype = (int)a.gate_up->bias_dtype; P.bias2_dtype = (int)a.down->bias_dtype;
    P.residual = a.residual; P.out = a.out; P.hf = (uint8_t *)hf; P.err = err;
    P.m = a.m; P.S = a.S; P.R = a.m * a.S; P.E = a.E; P.H = a.hidden; P.I = a.inter;
    P.g1 = a.hidden / a.gate_up->group_size; P.g2 = a.inter / a.down->group_size;
    P.gshift1 = log2_units(*a.gate_up); P.gshift2 = log2_units(*a.down);
    P.x_dtype = a.x_dtype; P.out_dtype = a.out_dtype; P.act = a.act;
    const int k1 = kind_of((int)a.gate_up->fmt, (int)a.gate_up->bits);
    const int k2 = kind_of((int)a.down->fmt, (int)a.down->bits);
    P.scale2_kind = k2 == K_NVFP4;
    P.down_affine = k2 == K_AFF4;
    const cudaError_t ce = k1 == K_AFF4    ? up_k<K_AFF4>(P, st)
                           : k1 == K_NVFP4 ? up_k<K_NVFP4>(P, st)
                                           : up_k<K_MXFP4>(P, st);
    if (ce != cudaSuccess) return ce;
    return k2 == K_AFF4    ? down_k<K_AFF4>(P, st)
           : k2 == K_NVFP4 ? down_k<K_NVFP4>(P, st)
                           : down_k<K_MXFP4>(P, st);
}

}  // namespace moe
