// mlp_few.cu -- the gated expert MLP for few tokens, in two kernels: what a decode
// step of one or a few sequences runs.
//
//   mlp_up    h[p] = act(G_e x_t) * (U_e x_t), times the pair's weight (and, NVFP4, the
//             down projection's scale2), split into bf16 planes in the workspace
//   mlp_down  out[t] = residual[t] + sum over the token's pairs of D_e h[p]
//
// Both are bound by the bytes of the weights that the tokens' experts hold, so each
// row of codes is read once for all pairs of its expert (up to the column blocks of
// a pass), straight from global memory into the lane that needs it, several steps
// ahead (cp.async into a ring that belongs to the lane: no barrier in the loop).
//
// The arithmetic runs on mma.sync m16n8k16 (bf16 operands, f32 sums): a tile is 16
// weight rows, the eight columns are x. That needs far fewer instructions a code
// than multiplying on the CUDA cores, does several pairs at the cost of one, and its
// 8-column shape wastes less here than tcgen05's 128-row tiles with one or two
// columns in use.
//   Codes are exact in bf16 (a 4-bit integer, an E2M1 value); scales are applied to
// f32 sums. A sum may then only run inside one scale group, while the four lanes
// that share a row each hold another unit of 32 codes (their 16-byte load). So a
// column belongs to one unit: lane q's x stands in column q alone and the other
// lanes are zero there, which keeps the four units' sums apart in four columns;
// the eight columns hold two sets (two pairs, or two planes of one pair).
//   x and h enter as sums of bf16 planes: bf16 one (exact), f16 two (exact), f32 and h
// for an f32 result three (24 bits), h for a 16-bit result two (16 bits, at least 8
// more than h rounded to bf16 would keep).
//   The affine bias needs the sum of x over each unit: an MMA with ones for A gives it
// in the accumulator's own layout.
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

// ------------------------------------------------------------------- codes

__device__ __forceinline__ uint32_t sub_bf16x2(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}
__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}

// Eight 4-bit codes of a word as bf16 pairs: p[i] = (code i, code i + 4).
// Integers: 0x4300 | c is 128 + c, exact, and the difference is exact. E2M1: sign
// and the three value bits land in bf16's sign, low exponent and top fraction bits,
// which is the value times 2^-126 (subnormals included); the product by 2^126 is exact.
template <int KIND>
__device__ __forceinline__ void expand(uint32_t w, uint32_t (&p)[4]) {
    if constexpr (KIND == K_AFF4) {
#pragma unroll
        for (int i = 0; i < 4; i++) p[i] = sub_bf16x2(((w >> (4 * i)) & 0x000F000Fu) | 0x43004300u, 0x43004300u);
    } else {
        const uint32_t v[4] = {((w << 12) & 0x80008000u) | ((w << 6) & 0x01C001C0u),
                               ((w << 8) & 0x80008000u) | ((w << 2) & 0x01C001C0u),
                               ((w << 4) & 0x80008000u) | ((w >> 2) & 0x01C001C0u),
                               (w & 0x80008000u) | ((w >> 6) & 0x01C001C0u)};
#pragma unroll
        for (int i = 0; i < 4; i++) p[i] = mul_bf16x2(v[i], 0x7E807E80u);
    }
}

__device__ __forceinline__ void mma(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                    uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Place of value c of a 32-value unit in the order of the B operand: register
// 4 (c / 8) + c % 4, half (c / 4) % 2, as expand() pairs the codes.
__device__ __forceinline__ uint32_t b_place(uint32_t c) { return 2u * (4u * (c >> 3) + (c & 3u)) + ((c >> 2) & 1u); }

// Scales of a row in shared memory for units u0 and u1 (element indices of the row).
template <int KIND> constexpr bool affine_kind = KIND == K_AFF4;

// Bytes of one row's scales.
__host__ __device__ inline uint32_t scale_bytes(int kind, uint32_t groups) {
    return kind == K_AFF4 ? groups * 2u : groups;
}

struct Sums {
    float xs[2];  // sums of x over the lane's two units (affine)
};

// One step of one tile: 16 rows x (4 units of 32 codes), all column blocks. wa, wb: the
// lane's unit of rows r and r + 8; sa, sb: those rows' scales (and biases ba, bb) in
// shared memory; u0: the first of the lane's two units in the accumulator's columns,
// u1 the second (both clamped to the row).
template <int KIND, int NBLK>
__device__ __forceinline__ void tile_step(const uint4 wa, const uint4 wb, const uint32_t (&B)[NBLK][16],
                                          const Sums (&xs)[NBLK], const uint8_t *sa, const uint8_t *sb,
                                          const uint8_t *ba, const uint8_t *bb, uint32_t u0, uint32_t u1,
                                          uint32_t gshift, float (&acc)[NBLK][2]) {
    const uint32_t a[4] = {wa.x, wa.y, wa.z, wa.w}, b[4] = {wb.x, wb.y, wb.z, wb.w};
    constexpr int PARTS = KIND == K_NVFP4 ? 2 : 1;  // scale groups in a unit
    float s[PARTS][4];                              // scale of (row r, u0), (r, u1), (r + 8, u0), (r + 8, u1)
    if constexpr (KIND == K_AFF4) {
        const uint32_t g0 = u0 >> gshift, g1 = u1 >> gshift;
        s[0][0] = bf16_bits_to_f32(((const unsigned short *)sa)[g0]);
        s[0][1] = bf16_bits_to_f32(((const unsigned short *)sa)[g1]);
        s[0][2] = bf16_bits_to_f32(((const unsigned short *)sb)[g0]);
        s[0][3] = bf16_bits_to_f32(((const unsigned short *)sb)[g1]);
    } else if constexpr (KIND == K_MXFP4) {
        s[0][0] = e8m0_to_f32(sa[u0]);
        s[0][1] = e8m0_to_f32(sa[u1]);
        s[0][2] = e8m0_to_f32(sb[u0]);
        s[0][3] = e8m0_to_f32(sb[u1]);
    } else {
        const uint32_t h[4] = {((const unsigned short *)sa)[u0], ((const unsigned short *)sa)[u1],
                               ((const unsigned short *)sb)[u0], ((const unsigned short *)sb)[u1]};
#pragma unroll
        for (int i = 0; i < 4; i++) {
            uint32_t f;  // two E4M3 bytes as f16 (exact)
            asm("{.reg .b16 h; cvt.u16.u32 h, %1; cvt.rn.f16x2.e4m3x2 %0, h;}" : "=r"(f) : "r"(h[i]));
            s[0][i] = f16_bits_to_f32(f & 0xFFFFu);
            s[PARTS - 1][i] = f16_bits_to_f32(f >> 16);
        }
    }
    float c[NBLK][4];
#pragma unroll
    for (int w = 0; w < 4; w++) {
        if (w % (4 / PARTS) == 0) {
#pragma unroll
            for (int n = 0; n < NBLK; n++) c[n][0] = c[n][1] = c[n][2] = c[n][3] = 0.f;
        }
        uint32_t pa[4], pb[4];
        expand<KIND>(a[w], pa);
        expand<KIND>(b[w], pb);
#pragma unroll
        for (int n = 0; n < NBLK; n++) {
            mma(c[n], pa[0], pb[0], pa[1], pb[1], B[n][4 * w], B[n][4 * w + 1]);
            mma(c[n], pa[2], pb[2], pa[3], pb[3], B[n][4 * w + 2], B[n][4 * w + 3]);
        }
        if (w % (4 / PARTS) == 4 / PARTS - 1) {
            const int h = w / (4 / PARTS);
#pragma unroll
            for (int n = 0; n < NBLK; n++) {
                acc[n][0] = fmaf(s[h][0], c[n][0], fmaf(s[h][1], c[n][1], acc[n][0]));
                acc[n][1] = fmaf(s[h][2], c[n][2], fmaf(s[h][3], c[n][3], acc[n][1]));
            }
        }
    }
    if constexpr (affine_kind<KIND>) {
        const uint32_t g0 = u0 >> gshift, g1 = u1 >> gshift;
        const float b0 = bf16_bits_to_f32(((const unsigned short *)ba)[g0]);
        const float b1 = bf16_bits_to_f32(((const unsigned short *)ba)[g1]);
        const float b2 = bf16_bits_to_f32(((const unsigned short *)bb)[g0]);
        const float b3 = bf16_bits_to_f32(((const unsigned short *)bb)[g1]);
#pragma unroll
        for (int n = 0; n < NBLK; n++) {
            acc[n][0] = fmaf(b0, xs[n].xs[0], fmaf(b1, xs[n].xs[1], acc[n][0]));
            acc[n][1] = fmaf(b2, xs[n].xs[0], fmaf(b3, xs[n].xs[1], acc[n][1]));
        }
    }
}

// Sums of x over the units of each column (affine): every row of A is ones.
template <int KIND, int NBLK>
__device__ __forceinline__ void unit_sums(const uint32_t (&B)[NBLK][16], Sums (&xs)[NBLK]) {
    if constexpr (affine_kind<KIND>) {
        constexpr uint32_t ONE = 0x3F803F80u;
#pragma unroll
        for (int n = 0; n < NBLK; n++) {
            float c[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int i = 0; i < 8; i++) mma(c, ONE, ONE, ONE, ONE, B[n][2 * i], B[n][2 * i + 1]);
            xs[n].xs[0] = c[0];
            xs[n].xs[1] = c[1];
        }
    }
}

// ------------------------------------------------------------------ routing

// The distinct valid experts of at most 256 pairs as bits, ascending ranks by prefix
// counts. All threads of the CTA call it; `mask` and `base` are shared arrays of 32.
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
    uint16_t *hf;                    // planes of h: [R][inter / 32][planes][32] bf16
    uint32_t *err;
    uint32_t m, R, S, E, H, I;       // H hidden, I inter
    uint32_t g1, g2, gshift1, gshift2;  // groups of a row; log2(units of 32 a group)
    int x_dtype, out_dtype, bias1_dtype, bias2_dtype, act, planes;
    int scale2_kind;                 // 1: the down projection is NVFP4 (scale2 in a2)
    uint32_t stages, slots, max_parts;  // ring depth; mlp_down: experts whose scales it holds, parts an expert
};

// Natural-order bf16 x of a unit (16 registers) in the order of the B operand.
__device__ __forceinline__ void permute_x(const uint32_t (&v)[16], uint32_t (&b)[16]) {
#pragma unroll
    for (int w = 0; w < 4; w++) {
        b[4 * w + 0] = __byte_perm(v[4 * w], v[4 * w + 2], 0x5410);
        b[4 * w + 1] = __byte_perm(v[4 * w], v[4 * w + 2], 0x7632);
        b[4 * w + 2] = __byte_perm(v[4 * w + 1], v[4 * w + 3], 0x5410);
        b[4 * w + 3] = __byte_perm(v[4 * w + 1], v[4 * w + 3], 0x7632);
    }
}

// Plane `plane` of two f32 values: bf16 of what the planes before it leave.
__device__ __forceinline__ uint32_t plane_of(float a, float b, uint32_t plane) {
    uint32_t p = 0;
    for (uint32_t i = 0; i <= plane; i++) {
        asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(p) : "f"(b), "f"(a));
        a -= __uint_as_float(p << 16);
        b -= __uint_as_float(p & 0xFFFF0000u);
    }
    return p;
}

// mlp_up. grid (inter / 32, ranks of distinct experts). A CTA holds 32 columns of h
// (64 weight rows: tile t pairs gate rows 8t..8t+7 with up rows 8t..8t+7, so that a
// lane's two accumulator rows are the gate and the up of one column) and its warps
// split hidden in steps of 128 codes.
template <int KIND, int XT, int NBLK>
__global__ void __launch_bounds__(FEW_THREADS, NBLK <= 2 ? 2 : 1) mlp_up(const FewParams P) {
    constexpr uint32_t PLANES = XT == DT_BF16 ? 1 : XT == DT_F16 ? 2 : 3;
    constexpr uint32_t SPP = PLANES == 3 ? 4 : PLANES;          // sets a pair (three planes: one left empty)
    constexpr uint32_t SETS = 2 * NBLK, PAIRS = SETS / SPP;     // of a pass
    constexpr uint32_t XB = XT == DT_F32 ? 8 : 4;               // 16-byte pieces of a unit of x
    constexpr uint32_t WBYTES = UP_TILES * 2 * 512, XBYTES = XB * 128;  // a stage of one warp
    constexpr uint32_t STAGE = WBYTES + NBLK * XBYTES;
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

    // scales (and affine biases) of the 64 rows: two blocks of 32 contiguous rows each
    const uint32_t c0 = blockIdx.x * 32u;
    const uint32_t srow = scale_bytes(KIND, P.g1);
    uint8_t *const s_s = sm + FEW_WARPS * P.stages * STAGE;
    uint8_t *const b_s = s_s + 64u * srow;
    const uint32_t sm0 = ptx::smem_u32(sm);
    for (uint32_t o = tid * 16u; o < 64u * srow; o += FEW_THREADS * 16u) {
        const uint32_t half = o >= 32u * srow;
        const size_t src = ((size_t)e * 2u * P.I + half * P.I + c0) * srow + (o - half * 32u * srow);
        ptx::cp_async_16(sm0 + (uint32_t)(s_s - sm) + o, P.s1 + src, 16);
        if constexpr (affine_kind<KIND>) ptx::cp_async_16(sm0 + (uint32_t)(b_s - sm) + o, P.a1 + src, 16);
    }
    ptx::cp_async_commit();
    __syncthreads();  // pairs[]

    const uint32_t r = lane >> 2, q = lane & 3u;
    const uint32_t nu = P.H / 32u, steps = (nu + 3u) / 4u;
    const uint32_t row_bytes = P.H / 2u;
    const bool active = ((lane >> 2) & 3u) == q;  // holds x of column lane / 4
    const uint32_t set0 = lane >> 4;              // its set of each block
    const uint32_t al = (lane >> 2) & 7u;         // its place among the active lanes
    const uint32_t ring = sm0 + warp * P.stages * STAGE;
    const uint8_t *const wg = P.w1 + ((size_t)e * 2u * P.I + c0 + r) * row_bytes;  // gate row of tile 0
    const size_t up = (size_t)P.I * row_bytes;
    const uint32_t n_mine = warp < steps ? (steps - warp + FEW_WARPS - 1u) / FEW_WARPS : 0u;

    for (uint32_t pb = 0; pb < np; pb += PAIRS) {
        const uint32_t npass = tmin<uint32_t>(PAIRS, np - pb);
        auto issue = [&](uint32_t i) {
            if (i < n_mine) {
                const uint32_t u = (warp + i * FEW_WARPS) * 4u + q;
                const uint32_t st = ring + (i % P.stages) * STAGE + lane * 16u;
                const bool in = u < nu;
                const uint8_t *src = wg + (in ? u : 0u) * 16u;
#pragma unroll
                for (uint32_t t = 0; t < UP_TILES; t++) {
                    ptx::cp_async_16(st + (2 * t) * 512u, src + (size_t)(8u * t) * row_bytes, in ? 16u : 0u);
                    ptx::cp_async_16(st + (2 * t + 1) * 512u, src + up + (size_t)(8u * t) * row_bytes, in ? 16u : 0u);
                }
                if (active) {
#pragma unroll
                    for (uint32_t n = 0; n < NBLK; n++) {
                        const uint32_t pi = (2u * n + set0) / SPP;
                        if (pi < npass) {
                            const size_t row = (size_t)(pairs[pb + pi] / P.S) * P.H + (in ? u : 0u) * 32u;
                            const uint8_t *xs = (const uint8_t *)P.x + row * (XT == DT_F32 ? 4u : 2u);
                            const uint32_t dst =
                                ring + (i % P.stages) * STAGE + WBYTES + n * XBYTES + al * 16u;
#pragma unroll
                            for (uint32_t k = 0; k < XB; k++)
                                ptx::cp_async_16(dst + k * 128u, xs + 16u * k, in ? 16u : 0u);
                        }
                    }
                }
            }
            ptx::cp_async_commit();
        };
        for (uint32_t i = 0; i < P.stages; i++) issue(i);
        if (pb == 0) {
            // the scales' group is the oldest; other threads' parts of them too
            if (P.stages == 2) asm volatile("cp.async.wait_group 2;" ::: "memory");
            else if (P.stages == 3) asm volatile("cp.async.wait_group 3;" ::: "memory");
            else asm volatile("cp.async.wait_group 4;" ::: "memory");
            __syncthreads();
        }
        float acc[UP_TILES][NBLK][2];
#pragma unroll
        for (uint32_t t = 0; t < UP_TILES; t++)
#pragma unroll
            for (int n = 0; n < NBLK; n++) acc[t][n][0] = acc[t][n][1] = 0.f;

        for (uint32_t i = 0; i < n_mine; i++) {
            if (P.stages == 2) asm volatile("cp.async.wait_group 1;" ::: "memory");
            else if (P.stages == 3) asm volatile("cp.async.wait_group 2;" ::: "memory");
            else asm volatile("cp.async.wait_group 3;" ::: "memory");
            const uint8_t *st = sm + warp * P.stages * STAGE + (i % P.stages) * STAGE;
            uint32_t B[NBLK][16];
#pragma unroll
            for (uint32_t n = 0; n < NBLK; n++) {
                const uint32_t set = 2u * n + set0;
                if (active && set / SPP < npass && set % SPP < PLANES) {
                    const uint4 *xp = (const uint4 *)(st + WBYTES + n * XBYTES + al * 16u);
                    uint32_t v[16];
                    if constexpr (XT == DT_F32) {
                        const uint32_t plane = set % 4u;
#pragma unroll
                        for (int k = 0; k < 8; k++) {
                            const uint4 f = xp[k * 8];
                            v[2 * k] = plane_of(__uint_as_float(f.x), __uint_as_float(f.y), plane);
                            v[2 * k + 1] = plane_of(__uint_as_float(f.z), __uint_as_float(f.w), plane);
                        }
                    } else {
#pragma unroll
                        for (int k = 0; k < 4; k++) {
                            const uint4 f = xp[k * 8];
                            v[4 * k] = f.x; v[4 * k + 1] = f.y; v[4 * k + 2] = f.z; v[4 * k + 3] = f.w;
                        }
                        if constexpr (XT == DT_F16) {
#pragma unroll
                            for (int k = 0; k < 16; k++)
                                v[k] = plane_of(f16_bits_to_f32(v[k] & 0xFFFFu), f16_bits_to_f32(v[k] >> 16), set % 2u);
                        }
                    }
                    permute_x(v, B[n]);
                } else {
#pragma unroll
                    for (int k = 0; k < 16; k++) B[n][k] = 0u;
                }
            }
            Sums xs[NBLK];
            unit_sums<KIND, NBLK>(B, xs);
            const uint32_t j = warp + i * FEW_WARPS;
            const uint32_t u0 = tmin<uint32_t>(4u * j + 2u * (q & 1u), nu - 1u), u1 = tmin<uint32_t>(u0 + 1u, nu - 1u);
#pragma unroll
            for (uint32_t t = 0; t < UP_TILES; t++) {
                const uint4 wa = *(const uint4 *)(st + (2 * t) * 512u + lane * 16u);
                const uint4 wb = *(const uint4 *)(st + (2 * t + 1) * 512u + lane * 16u);
                const uint32_t ra = (8u * t + r) * srow, rb = ra + 32u * srow;
                tile_step<KIND, NBLK>(wa, wb, B, xs, s_s + ra, s_s + rb, b_s + ra, b_s + rb, u0, u1, P.gshift1,
                                      acc[t]);
            }
            issue(i + P.stages);
        }
        asm volatile("cp.async.wait_all;" ::: "memory");
        __syncthreads();  // the ring is free: the warps' sums go there
        float *const red = (float *)sm;  // [warp][set][gate / up][32 columns]
#pragma unroll
        for (uint32_t t = 0; t < UP_TILES; t++)
#pragma unroll
            for (int n = 0; n < NBLK; n++)
#pragma unroll
                for (int h = 0; h < 2; h++) {
                    const float v = acc[t][n][h] + __shfl_xor_sync(FULL, acc[t][n][h], 1);
                    if (!(q & 1u)) red[((warp * SETS + 2u * n + (q >> 1)) * 2u + h) * 32u + 8u * t + r] = v;
                }
        __syncthreads();
        // one warp a pair: lane = column of h
        for (uint32_t pi = warp; pi < npass; pi += FEW_WARPS) {
            float g = 0.f, u = 0.f;
#pragma unroll
            for (uint32_t w = 0; w < FEW_WARPS; w++)
#pragma unroll
                for (uint32_t pl = 0; pl < PLANES; pl++) {
                    const uint32_t set = pi * SPP + pl;
                    g += red[((w * SETS + set) * 2u) * 32u + lane];
                    u += red[((w * SETS + set) * 2u + 1u) * 32u + lane];
                }
            const uint32_t p = pairs[pb + pi], c = c0 + lane;
            if constexpr (KIND == K_NVFP4) {
                const float s2 = __ldg((const float *)P.a1 + e);
                g *= s2;
                u *= s2;
            }
            const size_t bo = (size_t)e * 2u * P.I + c;
            g += load_bias(P.bias1, P.bias1_dtype, bo);
            u += load_bias(P.bias1, P.bias1_dtype, bo + P.I);
            float h = glu_act(P.act, g) * u * __ldg(P.weights + p);
            if (P.scale2_kind) h *= __ldg((const float *)P.a2 + e);
            uint16_t *dst = P.hf + ((size_t)p * (P.I / 32u) + blockIdx.x) * P.planes * 32u + b_place(lane);
            for (int pl = 0; pl < P.planes; pl++) {
                const __nv_bfloat16 b = __float2bfloat16_rn(h);
                dst[pl * 32] = __bfloat16_as_ushort(b);
                h -= __bfloat162float(b);
            }
        }
        __syncthreads();  // red is read before the next pass's copies land there
    }
}

// mlp_down. grid (hidden / 16): a CTA holds 16 columns of out. Its warps share the
// distinct experts (an expert's rows in PARTS strided parts where there are few),
// each keeps sums of its own for every token, added in warp order at the end: no
// atomics, one order. Weights and scales do not depend on mlp_up, so the ring's first
// stages are requested before waiting for it.
template <int KIND, int NPL, int NBLK>
__global__ void __launch_bounds__(FEW_THREADS, 2) mlp_down(const FewParams P) {
    constexpr uint32_t SPP = NPL == 3 ? 4 : 2, PAIRS = 2 * NBLK / SPP;  // sets a pair, pairs a pass
    constexpr uint32_t WBYTES = 2 * 512, HBYTES = 4 * 128, STAGE = WBYTES + NBLK * HBYTES;
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
    // items: (expert, part of its steps)
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

    const bool active = ((lane >> 2) & 3u) == q;
    const uint32_t set0 = lane >> 4, al = (lane >> 2) & 7u;

    // position of the copies and of the arithmetic in the warp's list of steps
    struct Pos {
        uint32_t item, ord, pb, j;  // item, its number in this warp, first pair, step
    };
    auto begin = [&]() {
        Pos p{warp, 0u, 0u, 0u};
        p.j = items ? warp % parts : 0u;
        return p;
    };
    auto advance = [&](Pos &p) {
        p.j += parts;
        if (p.j < steps) return;
        p.j = p.item % parts;
        p.pb += PAIRS;
        const uint32_t x = p.item / parts;
        if (p.pb < first[x + 1u] - first[x]) return;
        p.pb = 0u;
        p.item += FEW_WARPS;
        p.ord++;
        p.j = p.item % parts;
    };
    auto issue_w = [&](const Pos &p, uint32_t slot) {
        const uint32_t e = experts[p.item / parts];
        const uint32_t u = 4u * p.j + q;
        const bool in = u < nu;
        const uint8_t *src = P.w2 + ((size_t)e * P.H + row0 + r) * row_bytes + (in ? u : 0u) * 16u;
        const uint32_t st = ring + slot * STAGE + lane * 16u;
        ptx::cp_async_16(st, src, in ? 16u : 0u);
        ptx::cp_async_16(st + 512u, src + (size_t)8u * row_bytes, in ? 16u : 0u);
        if (p.pb == 0u && p.j == p.item % parts) {  // first step of the item: its scales
            const size_t so = ((size_t)e * P.H + row0) * srow;
            const uint32_t ss = sslots + (p.ord % P.slots) * sslot;
            for (uint32_t o = lane * 16u; o < 16u * srow; o += 512u) {
                ptx::cp_async_16(ss + o, P.s2 + so + o, 16);
                if constexpr (affine_kind<KIND>) ptx::cp_async_16(ss + 16u * srow + o, P.a2 + so + o, 16);
            }
        }
    };
    auto issue_h = [&](const Pos &p, uint32_t slot) {
        if (!active) return;
        const uint32_t x = p.item / parts, u = 4u * p.j + q;
        const bool in = u < nu;
#pragma unroll
        for (uint32_t n = 0; n < NBLK; n++) {
            const uint32_t set = 2u * n + set0;
            const uint32_t pi = p.pb + set / SPP, pl = set % SPP;
            if (pl < (uint32_t)NPL && pi < first[x + 1u] - first[x]) {
                const uint16_t *src =
                    P.hf + (((size_t)pairs[first[x] + pi] * nu + (in ? u : 0u)) * NPL + pl) * 32u;
                const uint32_t dst = ring + slot * STAGE + WBYTES + n * HBYTES + al * 16u;
#pragma unroll
                for (uint32_t k = 0; k < 4; k++) ptx::cp_async_16(dst + k * 128u, src + 8u * k, in ? 16u : 0u);
            }
        }
    };

    // `stages` steps ahead of the arithmetic, which P.slots covers: an item has at least
    // steps / max_parts steps
    Pos ahead = begin();
    uint32_t issued = 0;
    while (issued < P.stages && ahead.item < items) {
        issue_w(ahead, issued++);
        advance(ahead);
    }
    ptx::cp_async_commit();
    ptx::griddep_wait();  // h
    {
        Pos p = begin();
        for (uint32_t i = 0; i < P.stages; i++) {
            if (i < issued) {
                issue_h(p, i);
                advance(p);
            }
            ptx::cp_async_commit();
        }
    }

    Pos at = begin();
    float acc[NBLK][2];
#pragma unroll
    for (int n = 0; n < NBLK; n++) acc[n][0] = acc[n][1] = 0.f;
    uint32_t done = 0;
    while (at.item < items) {
        // the oldest stage has landed: `stages` groups follow the weights' first one
        switch (P.stages) {
            case 4: asm volatile("cp.async.wait_group 3;" ::: "memory"); break;
            case 6: asm volatile("cp.async.wait_group 5;" ::: "memory"); break;
            default: asm volatile("cp.async.wait_group 7;" ::: "memory"); break;
        }
        __syncwarp();  // and the other lanes' parts of the scales
        const uint32_t slot = done % P.stages;
        const uint32_t x = at.item / parts, cnt = first[x + 1u] - first[x];
        const uint8_t *st = wsm + slot * STAGE;
        uint32_t B[NBLK][16];
#pragma unroll
        for (uint32_t n = 0; n < NBLK; n++) {
            const uint32_t set = 2u * n + set0;
            const uint32_t pi = at.pb + set / SPP, pl = set % SPP;
            if (active && pl < (uint32_t)NPL && pi < cnt) {
                const uint4 *hp = (const uint4 *)(st + WBYTES + n * HBYTES + al * 16u);
#pragma unroll
                for (int k = 0; k < 4; k++) {
                    const uint4 f = hp[k * 8];
                    B[n][4 * k] = f.x; B[n][4 * k + 1] = f.y; B[n][4 * k + 2] = f.z; B[n][4 * k + 3] = f.w;
                }
            } else {
#pragma unroll
                for (int k = 0; k < 16; k++) B[n][k] = 0u;
            }
        }
        Sums xs[NBLK];
        unit_sums<KIND, NBLK>(B, xs);
        const uint32_t u0 = tmin<uint32_t>(4u * at.j + 2u * (q & 1u), nu - 1u), u1 = tmin<uint32_t>(u0 + 1u, nu - 1u);
        const uint8_t *ss = wsm + P.stages * STAGE + (at.ord % P.slots) * sslot;
        const uint4 wa = *(const uint4 *)(st + lane * 16u), wb = *(const uint4 *)(st + 512u + lane * 16u);
        tile_step<KIND, NBLK>(wa, wb, B, xs, ss + r * srow, ss + (r + 8u) * srow, ss + (16u + r) * srow,
                              ss + (24u + r) * srow, u0, u1, P.gshift2, acc);
        const Pos was = at;
        advance(at);
        done++;
        __syncwarp();  // every lane has read its stage and scales
        if (ahead.item < items) {
            issue_w(ahead, issued % P.stages);
            issue_h(ahead, issued % P.stages);
            issued++;
            advance(ahead);
        }
        ptx::cp_async_commit();
        if (at.pb != was.pb || at.item != was.item) {  // end of a pass: into the tokens' sums
#pragma unroll
            for (uint32_t n = 0; n < NBLK; n++)
#pragma unroll
                for (int h = 0; h < 2; h++) acc[n][h] += __shfl_xor_sync(FULL, acc[n][h], 1);
#pragma unroll
            for (uint32_t pi = 0; pi < PAIRS; pi++) {
                float v[2];
#pragma unroll
                for (int h = 0; h < 2; h++) {
                    // the planes of a pair: the two sets of its block, and the next block's first
                    float a = acc[pi * (SPP / 2)][h];
                    if constexpr (NPL == 3) {
                        if (q < 2u) a += acc[pi * 2 + 1][h];
                    }
                    v[h] = a + __shfl_xor_sync(FULL, a, 2);
                }
                if (q == 0u && was.pb + pi < cnt) {
                    float *y = ysm + ((size_t)warp * P.m + pairs[first[x] + was.pb + pi] / P.S) * 16u;
                    y[r] += v[0];
                    y[r + 8u] += v[1];
                }
            }
#pragma unroll
            for (int n = 0; n < NBLK; n++) acc[n][0] = acc[n][1] = 0.f;
            __syncwarp();
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

template <int KIND, int XT, int NBLK>
cudaError_t up_t(FewParams P, cudaStream_t st) {
    constexpr size_t stage = FEW_WARPS * (UP_TILES * 2 * 512 + NBLK * (XT == DT_F32 ? 8 : 4) * 128);
    const size_t scales = 64ull * scale_bytes(KIND, P.g1) * (KIND == K_AFF4 ? 2u : 1u);
    // as deep as two CTAs an SM (one with four blocks of columns) leave room for
    const size_t room = NBLK <= 2 && scales + 2 * stage <= FEW_SMEM_TWO ? FEW_SMEM_TWO : FEW_SMEM_ONE;
    P.stages = scales + 4 * stage <= room ? 4 : scales + 3 * stage <= room ? 3 : 2;
    const size_t smem = P.stages * stage + scales;
    auto kern = mlp_up<KIND, XT, NBLK>;
    static int smem_set[64];
    const cudaError_t e = ensure_dyn_smem(kern, smem, smem_set);
    if (e != cudaSuccess) return e;
    kern<<<dim3(P.I / 32u, tmin<uint32_t>(P.R, P.E)), FEW_THREADS, smem, st>>>(P);
    return cudaGetLastError();
}

template <int KIND, int NPL, int NBLK>
cudaError_t down_t(FewParams P, cudaStream_t st) {
    constexpr size_t stage = 2 * 512 + NBLK * 4 * 128;
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
    auto kern = mlp_down<KIND, NPL, NBLK>;
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

// Pairs of an expert that one pass takes: 1 for a single token, else the power of two
// above the mean when the pairs spread evenly, at least 2; more take further passes.
uint32_t pairs_a_pass(const FewParams &P) {
    if (P.m == 1) return 1;
    return P.R <= P.E ? 2u : P.R <= 2ull * P.E ? 4u : 8u;
}

template <int KIND, int XT>
cudaError_t up_x(const FewParams &P, cudaStream_t st) {
    constexpr uint32_t spp = XT == DT_BF16 ? 1 : XT == DT_F16 ? 2 : 4;
    const uint32_t blocks = (pairs_a_pass(P) * spp + 1u) / 2u;
    if constexpr (XT != DT_F32) {
        if (blocks <= 1) return up_t<KIND, XT, 1>(P, st);
    }
    if (blocks <= 2) return up_t<KIND, XT, 2>(P, st);
    return up_t<KIND, XT, 4>(P, st);
}

template <int KIND>
cudaError_t up_k(const FewParams &P, cudaStream_t st) {
    if (P.x_dtype == DT_F32) return up_x<KIND, DT_F32>(P, st);
    if (P.x_dtype == DT_BF16) return up_x<KIND, DT_BF16>(P, st);
    return up_x<KIND, DT_F16>(P, st);
}

template <int KIND>
cudaError_t down_k(const FewParams &P, cudaStream_t st) {
    const uint32_t n = pairs_a_pass(P);
    if (P.planes == 3) return n <= 1 ? down_t<KIND, 3, 2>(P, st) : down_t<KIND, 3, 4>(P, st);
    return n <= 1 ? down_t<KIND, 2, 1>(P, st) : n <= 2 ? down_t<KIND, 2, 2>(P, st) : down_t<KIND, 2, 4>(P, st);
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

int h_planes(int out_dtype) { return out_dtype == DT_F32 ? 3 : 2; }

}  // namespace

uint64_t mlp_few_workspace(uint32_t m, uint32_t inter, uint32_t S) {
    const uint64_t R = (uint64_t)m * S;
    return R <= FEW_MAX_R ? R * inter * 3ull * 2ull : 0ull;  // three bf16 planes of h
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
    // the deepest need of any variant: two stages with four blocks of f32 columns; four
    // stages with four blocks and six experts' scales
    const size_t up = 2ull * FEW_WARPS * (UP_TILES * 1024 + 4 * 1024) + sc1;
    const size_t dn = FEW_WARPS * (4ull * (1024 + 4 * 512) + 6ull * sc2) + 512ull * a.m;
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
    P.residual = a.residual; P.out = a.out; P.hf = (uint16_t *)hf; P.err = err;
    P.m = a.m; P.S = a.S; P.R = a.m * a.S; P.E = a.E; P.H = a.hidden; P.I = a.inter;
    P.g1 = a.hidden / a.gate_up->group_size; P.g2 = a.inter / a.down->group_size;
    P.gshift1 = log2_units(*a.gate_up); P.gshift2 = log2_units(*a.down);
    P.x_dtype = a.x_dtype; P.out_dtype = a.out_dtype; P.act = a.act; P.planes = h_planes(a.out_dtype);
    const int k1 = kind_of((int)a.gate_up->fmt, (int)a.gate_up->bits);
    const int k2 = kind_of((int)a.down->fmt, (int)a.down->bits);
    P.scale2_kind = k2 == K_NVFP4;
    const cudaError_t ce = k1 == K_AFF4    ? up_k<K_AFF4>(P, st)
                           : k1 == K_NVFP4 ? up_k<K_NVFP4>(P, st)
                                           : up_k<K_MXFP4>(P, st);
    if (ce != cudaSuccess) return ce;
    return k2 == K_AFF4    ? down_k<K_AFF4>(P, st)
           : k2 == K_NVFP4 ? down_k<K_NVFP4>(P, st)
                           : down_k<K_MXFP4>(P, st);
}

}  // namespace moe
