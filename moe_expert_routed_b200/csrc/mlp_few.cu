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
constexpr uint32_t UP_TILES = 4;         // tiles of a CTA's 64 rows
constexpr size_t FEW_SMEM_TWO = 110 * 1024, FEW_SMEM_ONE = 220 * 1024;  // two CTAs or one an SM

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

// From the pairs' step images at `base`; pairs at and past np are 0.
template <int KIND, int PLANES, int NB>
__device__ __forceinline__ void load_step(StepB<NB> &S, const uint8_t *base, uint32_t np, uint32_t lane) {
    constexpr uint32_t STRIDE = step_bytes(PLANES);
    const uint32_t q = lane & 3u;
    const bool active = ((lane >> 2) & 3u) == q;  // this lane's k of column lane / 4 are that column's unit
#pragma unroll
    for (uint32_t n = 0; n < NB; n++) {
        const uint32_t set = 2u * n + (lane >> 4), pair = set / PLANES, plane = set % PLANES;
        uint32_t(&b)[16] = S.b[n];
        if (active && pair < np) {
            const uint4 *v = (const uint4 *)(base + pair * STRIDE + plane * 256u + q * 64u);
#pragma unroll
            for (int i = 0; i < 4; i++) {
                const uint4 x = v[i];
                b[4 * i] = x.x; b[4 * i + 1] = x.y; b[4 * i + 2] = x.z; b[4 * i + 3] = x.w;
            }
        } else {
#pragma unroll
            for (int i = 0; i < 16; i++) b[i] = 0u;
        }
        // the lane's accumulator columns 2q, 2q + 1: units 2 (q mod 2) and the next of set 2n + q / 2
        const uint32_t cset = 2u * n + (q >> 1), cpair = cset / PLANES, cplane = cset % PLANES;
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
        if (cpair < np) v = *(const float4 *)(base + cpair * STRIDE + PLANES * 256u + (q & 1u) * 16u);
        const float unit = cplane ? code_unit<KIND> * 4.8828125e-4f : code_unit<KIND>;  // 2^-11
        S.f[n][0] = v.x * unit;
        S.f[n][1] = v.z * unit;
        S.xs[n][0] = cplane ? 0.f : v.y;  // the bias once a pair
        S.xs[n][1] = cplane ? 0.f : v.w;
    }
}

// 16 rows x 4 units: wa, wb the lane's unit of rows r and r + 8; sa, sb those rows' scales,
// ba, bb their biases; u0, u1 the units of the lane's accumulator columns.
template <int KIND, int NB>
__device__ __forceinline__ void tile_step(const uint4 wa, const uint4 wb, const StepB<NB> &S, const uint8_t *sa,
                                          const uint8_t *sb, const uint8_t *ba, const uint8_t *bb, uint32_t u0,
                                          uint32_t u1, uint32_t gshift, float (&acc)[NB][2]) {
    const uint32_t a[4] = {wa.x, wa.y, wa.z, wa.w}, b[4] = {wb.x, wb.y, wb.z, wb.w};
    constexpr int PARTS = KIND == K_NVFP4 ? 2 : 1;  // scale groups in a unit
    float s[PARTS][4];                              // of (row r, u0), (r, u1), (r + 8, u0), (r + 8, u1)
    if constexpr (KIND == K_AFF4) {
        const uint32_t g0 = u0 >> gshift, g1 = u1 >> gshift;
        s[0][0] = bf16_bits_to_f32(((const unsigned short *)sa)[g0]);
        s[0][2] = bf16_bits_to_f32(((const unsigned short *)sb)[g0]);
        s[0][1] = s[0][0];
        s[0][3] = s[0][2];
        if (gshift == 0u) {  // groups of one unit
            s[0][1] = bf16_bits_to_f32(((const unsigned short *)sa)[g1]);
            s[0][3] = bf16_bits_to_f32(((const unsigned short *)sb)[g1]);
        }
    } else if constexpr (KIND == K_MXFP4) {
        s[0][0] = e8m0_to_f32(sa[u0]);
        s[0][1] = e8m0_to_f32(sa[u1]);
        s[0][2] = e8m0_to_f32(sb[u0]);
        s[0][3] = e8m0_to_f32(sb[u1]);
    } else {
        from_e4m3x2(((const unsigned short *)sa)[u0], s[0][0], s[PARTS - 1][0]);
        from_e4m3x2(((const unsigned short *)sa)[u1], s[0][1], s[PARTS - 1][1]);
        from_e4m3x2(((const unsigned short *)sb)[u0], s[0][2], s[PARTS - 1][2]);
        from_e4m3x2(((const unsigned short *)sb)[u1], s[0][3], s[PARTS - 1][3]);
    }
    constexpr int WPP = 4 / PARTS;  // words a part
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
            acc[n][0] = fmaf(s[h][0], c[n][0] * S.f[n][0], fmaf(s[h][1], c[n][1] * S.f[n][1], acc[n][0]));
            acc[n][1] = fmaf(s[h][2], c[n][2] * S.f[n][0], fmaf(s[h][3], c[n][3] * S.f[n][1], acc[n][1]));
        }
    }
    if constexpr (affine_kind<KIND>) {
        const uint32_t g0 = u0 >> gshift, g1 = u1 >> gshift;
        float b0 = bf16_bits_to_f32(((const unsigned short *)ba)[g0]), b1 = b0;
        float b2 = bf16_bits_to_f32(((const unsigned short *)bb)[g0]), b3 = b2;
        if (gshift == 0u) {
            b1 = bf16_bits_to_f32(((const unsigned short *)ba)[g1]);
            b3 = bf16_bits_to_f32(((const unsigned short *)bb)[g1]);
        }
#pragma unroll
        for (int n = 0; n < NB; n++) {
            acc[n][0] = fmaf(b0, S.xs[n][0], fmaf(b1, S.xs[n][1], acc[n][0]));
            acc[n][1] = fmaf(b2, S.xs[n][0], fmaf(b3, S.xs[n][1], acc[n][1]));
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

// cp.async groups that may still be in flight.
__device__ __forceinline__ void wait_groups(uint32_t n) {
    switch (n) {
        case 1: asm volatile("cp.async.wait_group 1;" ::: "memory"); break;
        case 2: asm volatile("cp.async.wait_group 2;" ::: "memory"); break;
        case 3: asm volatile("cp.async.wait_group 3;" ::: "memory"); break;
        case 4: asm volatile("cp.async.wait_group 4;" ::: "memory"); break;
        case 5: asm volatile("cp.async.wait_group 5;" ::: "memory"); break;
        case 7: asm volatile("cp.async.wait_group 7;" ::: "memory"); break;
        default: asm volatile("cp.async.wait_group 0;" ::: "memory"); break;
    }
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
    uint32_t stages, slots, max_parts;  // ring depth; mlp_down: experts whose scales it holds, parts an expert
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
// column); its warps split hidden in steps of 128 codes.
template <int KIND, int XT, int NB>
__global__ void __launch_bounds__(FEW_THREADS, NB <= 2 ? 2 : 1) mlp_up(const FewParams P) {
    constexpr int PLANES = x_planes(XT), PP = 2 * NB / PLANES;  // pairs a pass
    constexpr uint32_t STAGE = UP_TILES * 2 * 512, XSTEP = step_bytes(PLANES);
    extern __shared__ __align__(16) uint8_t sm[];
    __shared__ uint32_t mask[32], base[33], wcount[FEW_WARPS], pairs[FEW_MAX_R], expert_s;

    const uint32_t tid = threadIdx.x, warp = tid >> 5, lane = tid & 31u;
    // mlp_down may start from here on: what came before this kernel is complete
    ptx::griddep_wait();
    ptx::griddep_launch_dependents();

    // the expert of this rank and its pairs, ascending
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
    const uint32_t e = expert_s;

    const uint32_t r = lane >> 2, q = lane & 3u;
    const uint32_t nu = P.H / 32u, steps = (nu + 3u) / 4u;
    const uint32_t row_bytes = P.H / 2u;
    const uint32_t c0 = blockIdx.x * 32u;
    const uint32_t srow = scale_bytes(KIND, P.g1);
    uint8_t *const xb = sm + FEW_WARPS * P.stages * STAGE + warp * PP * XSTEP;  // this warp's step images
    uint8_t *const s_s = sm + FEW_WARPS * (P.stages * STAGE + PP * XSTEP);
    uint8_t *const b_s = s_s + 64u * srow;
    const uint32_t sm0 = ptx::smem_u32(sm);
    const uint32_t ring = sm0 + warp * P.stages * STAGE + lane * 16u;
    const uint8_t *const wrow = P.w1 + ((size_t)e * 2u * P.I + c0 + r) * row_bytes + q * 16u;  // gate row of tile 0
    const size_t up = (size_t)P.I * row_bytes, trow = 8u * (size_t)row_bytes;
    const uint32_t n_mine = warp < steps ? (steps - warp + FEW_WARPS - 1u) / FEW_WARPS : 0u;

    // the weights of a step into the ring: this lane's unit of each of the 8 row groups
    const uint8_t *src = wrow;
    uint32_t ju = 0, is = 0;  // next step of this warp to request, its slot
    auto issue = [&]() {
        if (ju < n_mine) {
            const uint32_t u = (warp + ju * FEW_WARPS) * 4u + q, size = u < nu ? 16u : 0u;
            const uint8_t *g = size ? src : wrow;  // past the row: nothing is read, zeros are stored
            const uint32_t st = ring + is * STAGE;
#pragma unroll
            for (uint32_t t = 0; t < UP_TILES; t++, g += trow) {
                ptx::cp_async_16(st + (2 * t) * 512u, g, size);
                ptx::cp_async_16(st + (2 * t + 1) * 512u, g + up, size);
            }
            src += FEW_WARPS * 64u;
            is = is + 1u == P.stages ? 0u : is + 1u;
        }
        ju++;
        ptx::cp_async_commit();
    };
    auto restart = [&]() {
        src = wrow + warp * 64u;
        ju = is = 0u;
        for (uint32_t i = 0; i < P.stages; i++) issue();
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

    const uint32_t mine = __ballot_sync(FULL, valid && id == e);
    if (lane == 0) wcount[warp] = __popc(mine);
    __syncthreads();
    uint32_t np = 0, at = 0;
#pragma unroll
    for (uint32_t i = 0; i < FEW_WARPS; i++) {
        if (i < warp) at += wcount[i];
        np += wcount[i];
    }
    if (valid && id == e) pairs[at + __popc(mine & ((1u << lane) - 1u))] = tid;
    wait_groups(P.stages);  // the scales' group is the oldest
    __syncthreads();        // pairs[], and the other threads' parts of the scales

    for (uint32_t pb = 0; pb < np; pb += PP) {
        const uint32_t npass = tmin<uint32_t>(PP, np - pb);
        if (pb) restart();
        size_t xrow[PP];
        float4 xv[PP];
        auto fetch_x = [&](uint32_t i) {  // the lane's 4 values of each pair's step
            const uint32_t k = (warp + i * FEW_WARPS) * 128u + 4u * lane;
#pragma unroll
            for (uint32_t p = 0; p < PP; p++)
                xv[p] = p < npass && i < n_mine && k < P.H ? load_x4<XT>(P.x, xrow[p] + k)
                                                           : make_float4(0.f, 0.f, 0.f, 0.f);
        };
#pragma unroll
        for (uint32_t p = 0; p < PP; p++) xrow[p] = p < npass ? (size_t)(pairs[pb + p] / P.S) * P.H : 0u;
        fetch_x(0);
        float acc[UP_TILES][NB][2];
#pragma unroll
        for (uint32_t t = 0; t < UP_TILES; t++)
#pragma unroll
            for (int n = 0; n < NB; n++) acc[t][n][0] = acc[t][n][1] = 0.f;

        const uint8_t *st = sm + warp * P.stages * STAGE + lane * 16u;
        uint32_t slot = 0;
        for (uint32_t i = 0; i < n_mine; i++) {
#pragma unroll
            for (uint32_t p = 0; p < PP; p++)
                if (p < npass) write_step<KIND, PLANES>(xb + p * XSTEP, xv[p], lane);
            __syncwarp();
            StepB<NB> B;
            load_step<KIND, PLANES, NB>(B, xb, npass, lane);
            __syncwarp();  // read before the next step's image is written
            fetch_x(i + 1u);
            wait_groups(P.stages - 1u);
            const uint32_t u = 4u * (warp + i * FEW_WARPS) + 2u * (q & 1u);
            const uint32_t u0 = tmin<uint32_t>(u, nu - 1u), u1 = tmin<uint32_t>(u + 1u, nu - 1u);
            const uint8_t *w = st + slot * STAGE;
            uint32_t so = r * srow;
#pragma unroll
            for (uint32_t t = 0; t < UP_TILES; t++, so += 8u * srow)
                tile_step<KIND, NB>(*(const uint4 *)(w + 2 * t * 512), *(const uint4 *)(w + (2 * t + 1) * 512), B,
                                    s_s + so, s_s + so + 32u * srow, b_s + so, b_s + so + 32u * srow, u0, u1,
                                    P.gshift1, acc[t]);
            slot = slot + 1u == P.stages ? 0u : slot + 1u;
            issue();
        }
        asm volatile("cp.async.wait_all;" ::: "memory");
        __syncthreads();  // the ring is free: the warps' sums go there
        float *const red = (float *)sm;  // [warp][pair][gate / up][32 columns]
#pragma unroll
        for (uint32_t t = 0; t < UP_TILES; t++)
#pragma unroll
            for (int n = 0; n < NB; n++)
#pragma unroll
                for (int h = 0; h < 2; h++) {
                    float v = acc[t][n][h];
                    v += __shfl_xor_sync(FULL, v, 1);
                    if constexpr (PLANES == 2) v += __shfl_xor_sync(FULL, v, 2);
                    if (PLANES == 2 ? q == 0u : !(q & 1u)) {
                        const uint32_t p = PLANES == 2 ? n : 2u * n + (q >> 1);
                        red[((warp * PP + p) * 2u + h) * 32u + 8u * t + r] = v;
                    }
                }
        __syncthreads();
        // one warp a pair: lane = column of h
        for (uint32_t pi = warp; pi < npass; pi += FEW_WARPS) {
            float g = 0.f, v = 0.f;
#pragma unroll
            for (uint32_t w = 0; w < FEW_WARPS; w++) {
                g += red[((w * PP + pi) * 2u) * 32u + lane];
                v += red[((w * PP + pi) * 2u + 1u) * 32u + lane];
            }
            const uint32_t p = pairs[pb + pi], c = c0 + lane;
            if constexpr (KIND == K_NVFP4) {
                const float s2 = __ldg((const float *)P.a1 + e);
                g *= s2;
                v *= s2;
            }
            const size_t bo = (size_t)e * 2u * P.I + c;
            g += load_bias(P.bias1, P.bias1_dtype, bo);
            v += load_bias(P.bias1, P.bias1_dtype, bo + P.I);
            float h = glu_act(P.act, g) * v * __ldg(P.weights + p);
            if (P.scale2_kind) h *= __ldg((const float *)P.a2 + e);
            // this unit of the pair's step image
            const int planes = h_planes(P.out_dtype);
            const uint32_t iu = P.I / 32u, un = blockIdx.x & 3u;
            uint8_t *img = P.hf + ((size_t)p * ((iu + 3u) / 4u) + (blockIdx.x >> 2)) * step_bytes(planes);
            const float sum = [&] {
                float s = h;
#pragma unroll
                for (int d = 16; d > 0; d >>= 1) s += __shfl_xor_sync(FULL, s, d);
                return s;
            }();
            float scale, factor;
            unit_scale(__reduce_max_sync(FULL, __float_as_uint(h) & 0x7FFFFFFFu), scale, factor);
            h *= scale;
            if (b_sixteenth(P.down_affine, lane)) h *= 0.0625f;
            uint16_t *dst = (uint16_t *)(img + un * 64u) + b_place(P.down_affine, lane);
            for (int k = 0; k < planes; k++, dst += 128) {
                const __half b = __float2half_rn(h);
                *dst = __half_as_ushort(b);
                h = (h - __half2float(b)) * 2048.f;
            }
            float2 *fs = (float2 *)(img + planes * 256);
            if (lane == 0) fs[un] = make_float2(factor, sum);
            // units past inter in the last step are zero
            if (blockIdx.x + 1u == iu)
                for (uint32_t z = un + 1u; z < 4u; z++) {
                    for (int k = 0; k < planes; k++) ((uint16_t *)(img + k * 256 + z * 64u))[lane] = 0;
                    if (lane == 0) fs[z] = make_float2(0.f, 0.f);
                }
        }
        __syncthreads();  // red is read before the next pass's copies land there
    }
}

// mlp_down. grid (hidden / 16): a CTA holds 16 columns of out. Its warps share the
// distinct experts (an expert's rows in strided parts where there are few), each keeps
// sums of its own for every token, added in warp order at the end: no atomics, one
// order. Weights and scales do not depend on mlp_up, so the ring's first stages are
// requested before waiting for it.
template <int KIND, int NPL, int NB>
__global__ void __launch_bounds__(FEW_THREADS, 2) mlp_down(const FewParams P) {
    constexpr uint32_t PP = 2 * NB / NPL;  // pairs a pass
    constexpr uint32_t HSTEP = step_bytes(NPL), WBYTES = 2 * 512, STAGE = WBYTES + PP * HSTEP;
    extern __shared__ __align__(16) uint8_t sm[];
    __shared__ uint32_t mask[32], base[33], ids_s[FEW_MAX_R], first[FEW_MAX_R + 1], pairs[FEW_MAX_R],
        experts[FEW_MAX_R];

    const uint32_t tid = threadIdx.x, warp = tid >> 5, lane = tid & 31u;
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

    const uint32_t r = lane >> 2, q = lane & 3u;
    const uint32_t nu = P.I / 32u, steps = (nu + 3u) / 4u, row_bytes = P.I / 2u;
    const uint32_t row0 = blockIdx.x * 16u;
    const uint32_t srow = scale_bytes(KIND, P.g2), sslot = 16u * srow * (affine_kind<KIND> ? 2u : 1u);
    // items: (expert, part of its steps), dealt to the warps in turn
    const uint32_t parts = D == 0 || D % FEW_WARPS == 0 || D >= 32u
                               ? 1u
                               : tmin<uint32_t>(D >= FEW_WARPS ? 2u : FEW_WARPS / D, P.max_parts);
    const uint32_t items = D * parts;
    const uint32_t warp_bytes = P.stages * STAGE + P.slots * sslot;
    uint8_t *const wsm = sm + warp * warp_bytes;
    const uint32_t ring = ptx::smem_u32(wsm), sslots = ring + P.stages * STAGE;
    float *const ysm = (float *)(sm + FEW_WARPS * warp_bytes);  // [warp][token][16]
    for (uint32_t o = tid; o < FEW_WARPS * P.m * 16u; o += FEW_THREADS) ysm[o] = 0.f;
    __syncthreads();

    // a position in the warp's list of steps; x, j0: the item's expert and first step
    struct Pos {
        uint32_t item, slot, x, j0, pb, j, cnt, first;
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
    auto advance = [&](Pos &p) {
        p.j += parts;
        if (p.j < steps) return false;
        p.j = p.j0;
        p.pb += PP;
        if (p.pb >= p.cnt) {
            p.item += FEW_WARPS;
            p.slot = p.slot + 1u == P.slots ? 0u : p.slot + 1u;
            enter(p);
        }
        return true;  // a pass ended
    };
    auto issue_w = [&](const Pos &p, uint32_t stage) {
        const uint32_t e = experts[p.x];
        const size_t row = (size_t)e * P.H + row0;
        const uint32_t u = 4u * p.j + q, size = u < nu ? 16u : 0u;
        const uint8_t *src = P.w2 + (row + r) * row_bytes + (size ? u : 0u) * 16u;
        const uint32_t st = ring + stage * STAGE + lane * 16u;
        ptx::cp_async_16(st, src, size);
        ptx::cp_async_16(st + 512u, src + 8u * row_bytes, size);
        if (p.pb == 0u && p.j == p.j0) {  // first step of the item: its scales
            const uint32_t ss = sslots + p.slot * sslot;
            for (uint32_t o = lane * 16u; o < 16u * srow; o += 512u) {
                ptx::cp_async_16(ss + o, P.s2 + row * srow + o, 16);
                if constexpr (affine_kind<KIND>) ptx::cp_async_16(ss + 16u * srow + o, P.a2 + row * srow + o, 16);
            }
        }
    };
    auto issue_h = [&](const Pos &p, uint32_t stage) {
        const uint32_t st = ring + stage * STAGE + WBYTES;
#pragma unroll
        for (uint32_t k = 0; k < PP; k++) {
            if (p.pb + k < p.cnt) {
                const uint8_t *src = P.hf + ((size_t)pairs[p.first + p.pb + k] * steps + p.j) * HSTEP;
                for (uint32_t o = lane * 16u; o < HSTEP; o += 512u) ptx::cp_async_16(st + k * HSTEP + o, src + o, 16);
            }
        }
    };

    // `stages` steps ahead of the arithmetic, which P.slots covers: an item has at least
    // steps / max_parts steps
    Pos ahead{};
    ahead.item = warp;
    enter(ahead);
    Pos at = ahead, fill = ahead;
    uint32_t issued = 0;
    while (issued < P.stages && ahead.item < items) {
        issue_w(ahead, issued++);
        advance(ahead);
    }
    ptx::cp_async_commit();
    ptx::griddep_wait();  // h
    for (uint32_t i = 0; i < P.stages; i++) {
        if (i < issued) {
            issue_h(fill, i);
            advance(fill);
        }
        ptx::cp_async_commit();
    }

    float acc[NB][2];
#pragma unroll
    for (int n = 0; n < NB; n++) acc[n][0] = acc[n][1] = 0.f;
    uint32_t stage = 0;
    while (at.item < items) {
        wait_groups(P.stages - 1u);  // the oldest stage: its weights came in an older group
        __syncwarp();                // and the other lanes' parts of the scales and of h
        const uint8_t *st = wsm + stage * STAGE;
        StepB<NB> B;
        load_step<KIND, NPL, NB>(B, st + WBYTES, at.cnt - at.pb, lane);
        const uint32_t u = 4u * at.j + 2u * (q & 1u);
        const uint32_t u0 = tmin<uint32_t>(u, nu - 1u), u1 = tmin<uint32_t>(u + 1u, nu - 1u);
        const uint8_t *ss = wsm + P.stages * STAGE + at.slot * sslot + r * srow;
        tile_step<KIND, NB>(*(const uint4 *)(st + lane * 16u), *(const uint4 *)(st + 512u + lane * 16u), B, ss,
                            ss + 8u * srow, ss + 16u * srow, ss + 24u * srow, u0, u1, P.gshift2, acc);
        const uint32_t pfirst = at.first + at.pb, pcnt = at.cnt - at.pb;
        const bool ended = advance(at);
        __syncwarp();  // every lane has read its stage and scales
        if (ahead.item < items) {
            issue_w(ahead, stage);
            issue_h(ahead, stage);
            advance(ahead);
        }
        ptx::cp_async_commit();
        stage = stage + 1u == P.stages ? 0u : stage + 1u;
        if (ended) {  // end of a pass: into the tokens' sums
#pragma unroll
            for (uint32_t n = 0; n < NB; n++) {
                float v[2];
#pragma unroll
                for (int h = 0; h < 2; h++) {
                    v[h] = acc[n][h] + __shfl_xor_sync(FULL, acc[n][h], 1);
                    if constexpr (NPL == 2) v[h] += __shfl_xor_sync(FULL, v[h], 2);
                    acc[n][h] = 0.f;
                }
                // one pair at a time: two of them may be one token's
#pragma unroll
                for (uint32_t k = 0; k < 2u / NPL; k++) {
                    const uint32_t p = n * (2u / NPL) + k;
                    if (q == 2u * k && p < pcnt) {
                        float *y = ysm + ((size_t)warp * P.m + pairs[pfirst + p] / P.S) * 16u;
                        y[r] += v[0];
                        y[r + 8u] += v[1];
                    }
                    __syncwarp();
                }
            }
        }
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
    __syncthreads();
    for (uint32_t o = tid; o < P.m * 16u; o += FEW_THREADS) {
        const uint32_t t = o >> 4, c = row0 + (o & 15u);
        float y = 0.f;
#pragma unroll
        for (uint32_t w = 0; w < FEW_WARPS; w++) y += ysm[((size_t)w * P.m + t) * 16u + (o & 15u)];
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
}

// ------------------------------------------------------------------ launches

template <int KIND, int XT, int NB>
cudaError_t up_t(FewParams P, cudaStream_t st) {
    constexpr size_t stage = FEW_WARPS * UP_TILES * 2 * 512;
    constexpr size_t image = FEW_WARPS * (2 * NB / x_planes(XT)) * step_bytes(x_planes(XT));
    const size_t fixed = image + 64ull * scale_bytes(KIND, P.g1) * (KIND == K_AFF4 ? 2u : 1u);
    // as deep as two CTAs an SM leave room for
    const size_t room = fixed + 2 * stage <= FEW_SMEM_TWO ? FEW_SMEM_TWO : FEW_SMEM_ONE;
    P.stages = fixed + 4 * stage <= room ? 4 : fixed + 3 * stage <= room ? 3 : 2;
    const size_t smem = P.stages * stage + fixed;
    auto kern = mlp_up<KIND, XT, NB>;
    static int smem_set[64];
    const cudaError_t e = ensure_dyn_smem(kern, smem, smem_set);
    if (e != cudaSuccess) return e;
    kern<<<dim3(P.I / 32u, tmin<uint32_t>(P.R, P.E)), FEW_THREADS, smem, st>>>(P);
    return cudaGetLastError();
}

template <int KIND, int NPL, int NB>
cudaError_t down_t(FewParams P, cudaStream_t st) {
    constexpr size_t stage = 2 * 512 + (2 * NB / NPL) * step_bytes(NPL);
    const size_t sslot = 16ull * scale_bytes(KIND, P.g2) * (KIND == K_AFF4 ? 2u : 1u);
    const uint32_t steps = (P.I / 32u + 3u) / 4u;
    P.max_parts = steps / 3u ? steps / 3u : 1u;
    const uint32_t least = steps / P.max_parts;  // steps of an item
    size_t smem = 0;
    for (uint32_t stages = 8;; stages -= 2) {
        P.stages = stages;
        P.slots = stages / least + 2u;
        smem = FEW_WARPS * (P.stages * stage + P.slots * sslot) + 512ull * P.m;
        if (smem <= FEW_SMEM_TWO || stages == 4u) break;
    }
    auto kern = mlp_down<KIND, NPL, NB>;
    static int smem_set[64];
    const cudaError_t e = ensure_dyn_smem(kern, smem, smem_set);
    if (e != cudaSuccess) return e;
    // a programmatic dependent of mlp_up: it requests its weights while mlp_up runs and
    // waits (griddepcontrol.wait) before it reads h
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(P.H / 16u);
    cfg.blockDim = dim3(FEW_THREADS);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
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
    switch (blocks_a_pass(P, x_planes(XT))) {
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
    switch (blocks_a_pass(P, NPL)) {
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
// projections, at most 256 pairs of at most 64 tokens, scales of a CTA's rows that fit
// in shared memory beside the ring.
bool mlp_few_supported(const MlpArgs &a) {
    const uint64_t R = (uint64_t)a.m * a.S;
    if (R > FEW_MAX_R || a.m > FEW_MAX_TOKENS || a.E > MOE_ROUTE_MAX_EXPERTS) return false;
    if (!projection_ok(*a.gate_up, a.hidden) || !projection_ok(*a.down, a.inter)) return false;
    if ((uintptr_t)a.x & 15u) return false;
    const int k1 = kind_of((int)a.gate_up->fmt, (int)a.gate_up->bits);
    const int k2 = kind_of((int)a.down->fmt, (int)a.down->bits);
    const size_t sc1 = 64ull * scale_bytes(k1, a.hidden / a.gate_up->group_size) * (k1 == K_AFF4 ? 2u : 1u);
    const size_t sc2 = 16ull * scale_bytes(k2, a.inter / a.down->group_size) * (k2 == K_AFF4 ? 2u : 1u);
    // the least that the widest variants need: two stages; four stages, six experts' scales
    const size_t up = FEW_WARPS * (2ull * UP_TILES * 1024 + 8ull * step_bytes(1)) + sc1;
    const size_t dn = FEW_WARPS * (4ull * (1024 + 8ull * step_bytes(1)) + 6ull * sc2) + 512ull * a.m;
    return up <= FEW_SMEM_ONE && dn <= FEW_SMEM_ONE;
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
