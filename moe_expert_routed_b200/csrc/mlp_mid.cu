// mlp_mid.cu -- the gated expert MLP for some tens of pairs an expert: a block of
// tokens, a batch of sequences. Two grouped products on mma.sync over the routing's tiles
// of up to 24 pairs,
//   mid_product<UP>    h[p] = act(G_e x_t) * (U_e x_t)
//   mid_product<DOWN>  z[p] = weight[p] * D_e h[p]
// and the sum of z (weighted first: small weights keep z in f32's range where h is large).
//
// With so few columns a 128-row tcgen05 tile is bound by what hands it the dequantised
// operand, stage by stage, not by its arithmetic; here codes go from shared memory to the
// registers that the MMA reads. As in mlp_few.cu (operands and images are its own) the
// codes stay exact f16 values and scales are applied to f32 sums of a unit of 32, so no
// weight is rounded. Here all eight columns of an MMA are pairs: the four lanes of a row
// take a quarter of the same unit each (of the same scale's 16 codes, NVFP4).
//
// x is scaled by one power of two a token, h by one a unit; both are one f16 plane: exact
// for bf16 x down to 2^-31 of the token's largest value and for f16 x down to 2^-28 (2^-27
// and 2^-24 where x meets 16-fold codes), off by at most 2^-39 (2^-35) of it below; 11 bits
// of h, whose rounding adds no more to a 16-bit result than its own does (f16: 2.9e-4
// against 64 bits instead of 2.1e-4; bf16: nothing to be seen). f32 types take the other ways.
//
// A CTA: 128 weight rows, 32 a warp as two tiles, which share the registers of x; three to
// five CTAs an SM. Steps of 128 codes come by cp.async into a ring of two or three stages,
// one barrier a step. Eight warps a CTA, two CTAs an SM: 338 us against 322 (256 tokens,
// 3-bit codebook), 264 against 238 (NVFP4). 24 pairs a tile leave the registers for five
// CTAs: 242 us against 260 with tiles of 32 and four (affine 4 bits), 221 against 232.
// Bound by instructions: for each unit and 32 rows 40 (affine 4 bits) to 90 (3-bit codebook)
// to expand and scale the codes, 20 for each block of 8 pairs, 30 for copies and scales; the
// scheduler issues in 54 to 57 % of its cycles, the ALU is busy for 49 %, MMA for 20 %. With no
// products at all 142 of (then) 322 us are left: each CTA's chain of dependent loads and its
// empty ring.
// 128 experts of 2,816 x 704, top-8, 256 tokens: 281 us (3-bit codebook; the tcgen05 grouped
// products 558), 224 (affine 4 bits; 554), 202 (NVFP4; 389), 247 (affine 8 bits; 561).
#include "cb3_blocks.h"
#include "common.cuh"
#include "internal.h"
#include "mlp_codes.cuh"
#include "ptx.cuh"

namespace moe {
namespace {

constexpr uint32_t MID_WARPS = 4;
constexpr uint32_t MID_THREADS = 32 * MID_WARPS, MID_ROWS = 32 * MID_WARPS, MID_BLOCKS = 3;
constexpr uint32_t MID_PAIRS = 8 * MID_BLOCKS;  // of a tile
// Affine codes are f16 integers times 2^-24; the sums of x that meet the biases are scaled
// alike, and the results back.
constexpr float CODE_UNIT = 16777216.f;

// Bytes of a row's 128 codes in a stage: padded so that the lanes' quarters of eight rows
// lie in different banks (3 bits: the 16-byte blocks that hold 14 words of 10 codes; 6 bits: two lanes can meet).
__host__ __device__ constexpr uint32_t line(int m) {
    return m == M_A8 ? 160u : m == M_A6 ? 112u : m == M_CB2 ? 48u : 80u;
}
// A pair's 128 values of x or h in a stage (read 16 bytes a lane; NVFP4 8).
__host__ __device__ constexpr uint32_t x_line(int m) { return m == M_NV ? 288u : 320u; }
__host__ __device__ constexpr uint32_t stage_bytes(int m) {
    return MID_ROWS * line(m) + MID_PAIRS * (x_line(m) + 32u);
}
// CTAs an SM: five where their registers hold the expansion (tables of a codebook spill:
// 326 us against 304 with four), as many as the stages leave room for.
__host__ __device__ constexpr uint32_t ctas(int m) { return m == M_A8 ? 3u : m == M_A6 || codebook(m) ? 4u : 5u; }
__host__ __device__ constexpr uint32_t ring(int m) {
    return 3u * stage_bytes(m) <= 228u * 1024u / ctas(m) - 1024u ? 3u : 2u;
}
constexpr uint32_t HC = 16 * MID_WARPS, HB = HC + 4;  // UP: columns of h, floats of a pair's in the epilogue

struct MidParams {
    const uint8_t *w, *s, *a;    // packed codes, scales, affine biases or scale2 (or codebook)
    const void *bias;            // expert biases, or null
    const uint8_t *x;            // images: [token] (UP), [place among the sorted pairs] (DOWN)
    const float *factor;         // UP: of the tokens' values
    const float *weights;        // DOWN: of the pairs
    const uint32_t *offsets, *sorted_pairs, *tiles, *tile_count;
    void *out;                   // UP: images of h by sorted place; DOWN: z [pair][n] f32
    uint32_t k, n, S;            // n: rows of out (UP: of gate, the up rows follow)
    uint32_t row_bytes, groups, gshift;
    int bias_dtype, act, order;  // order of h's values in its images
    int sums;                    // UP: the down projection is affine and needs sums of h
};

// Two f32 values in one 64-bit register pair.
__device__ __forceinline__ uint64_t pack2(float a, float b) {
    uint64_t d;
    asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "f"(a), "f"(b));
    return d;
}
__device__ __forceinline__ float2 unpack2(uint64_t v) {
    float2 d;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(d.x), "=f"(d.y) : "l"(v));
    return d;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
    uint64_t d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}

__device__ __forceinline__ uint64_t lds64x(uint32_t a) {
    uint64_t v;
    asm volatile("ld.shared.b64 %0, [%1];" : "=l"(v) : "r"(a));
    return v;
}

// This lane's 8 codes of a unit from its row's line: quarter q, or (NVFP4) four of each
// scale's 16; `code`: 3-bit codes before the quarter in the line.
template <int MODE>
__device__ __forceinline__ void quarter(uint32_t at, uint32_t u, uint32_t q, uint32_t code, uint32_t (&w)[words(MODE)]) {
    if constexpr (MODE == M_NV) {
        w[0] = lds16(at + u * 16u + q * 2u) | lds16(at + u * 16u + 8u + q * 2u) << 16;
    } else if constexpr (MODE == M_A8) {
        const uint2 v = lds64(at + u * 32u + q * 8u);
        w[0] = v.x; w[1] = v.y;
    } else if constexpr (MODE == M_A6) {
        const uint32_t p = at + u * 24u + q * 6u;
        w[0] = lds16(p) | lds16(p + 2u) << 16;
        w[1] = lds16(p + 4u);
    } else if constexpr (MODE == M_CB2) {
        w[0] = lds16(at + u * 8u + q * 2u);
    } else if constexpr (MODE == M_CB3) {
        const uint32_t word = code * 205u >> 11;  // code / 10 (codes below 138)
        // 30 bits of the first word, then the next one's
        w[0] = __funnelshift_r(lds32(at + word * 4u) << 2, lds32(at + word * 4u + 4u), 3u * (code - 10u * word) + 2u);
    } else {
        w[0] = lds32(at + u * 16u + q * 4u);
    }
}

// A unit's scale as it is stored (NVFP4: two), and as f32.
template <int MODE>
__device__ __forceinline__ uint32_t raw_scale(const uint8_t *p) {
    // volatile: requested where it stands, a step ahead of its use
    uint32_t v;
    if constexpr (MODE == M_MX) asm volatile("ld.global.nc.u8 %0, [%1];" : "=r"(v) : "l"(p));
    else asm volatile("ld.global.nc.u16 %0, [%1];" : "=r"(v) : "l"(p));
    return v;
}
template <int MODE>
__device__ __forceinline__ float scale_f32(uint32_t v) {
    if constexpr (affine(MODE)) return bf16_bits_to_f32(v);
    else if constexpr (codebook(MODE)) return f16_bits_to_f32(v);
    else return e8m0_to_f32(v);
}

// The warp's 32 rows x a step x 8 NT pairs; past the last column codes and x are zero. row: shared address of the
// lane's first row, xs, fs: of its part of the pairs' values, and of their factors and sums; c0: 3-bit codes
// before the step in the line; raw, rawb: unit q's scales of the lane's four
// rows, two in a register.
template <int MODE, bool UP, int NT>
__device__ __forceinline__ void mid_step(uint32_t row, uint32_t xs, uint32_t fs, uint32_t c0,
                                         const uint32_t (&raw)[2], const uint32_t (&rawb)[2], const Table<MODE> &tab,
                                         uint32_t lane, uint64_t (&acc)[2][2][MID_BLOCKS]) {
    const uint32_t q = lane & 3u;
#pragma unroll
    for (uint32_t u = 0; u < 4; u++) {
        uint32_t p[4][4];
        uint64_t s[4], s1[MODE == M_NV ? 4 : 1], b[affine(MODE) ? 4 : 1];
        uint32_t sv[2], bv[2];
#pragma unroll
        for (uint32_t t = 0; t < 2; t++) {
            sv[t] = __shfl_sync(FULL, raw[t], (lane & ~3u) | u);
            if constexpr (affine(MODE)) bv[t] = __shfl_sync(FULL, rawb[t], (lane & ~3u) | u);
        }
#pragma unroll
        for (uint32_t i = 0; i < 4; i++) {
            uint32_t w[words(MODE)];
            quarter<MODE>(row + 8u * i * line(MODE), u, q, c0 + 32u * u + 8u * q, w);
            expand<MODE, false>(w, 0, tab, p[i]);
            const uint32_t v = i & 1u ? sv[i >> 1] >> 16 : sv[i >> 1] & 0xFFFFu;
            if constexpr (MODE == M_NV) {
                float f0, f1;
                from_e4m3x2(v, f0, f1);
                s[i] = pack2(f0, f0);
                s1[i] = pack2(f1, f1);
            } else {
                const float f = scale_f32<MODE>(v);
                s[i] = pack2(f, f);
            }
            if constexpr (affine(MODE)) {
                const float f = __uint_as_float(i & 1u ? bv[i >> 1] & 0xFFFF0000u : bv[i >> 1] << 16);
                b[i] = pack2(f, f);
            }
        }
#pragma unroll
        for (uint32_t n = 0; n < NT; n++) {
            uint4 B;
            if constexpr (MODE == M_NV) {
                const uint2 lo = lds64(xs + n * 8u * x_line(MODE) + u * 64u);
                const uint2 hi = lds64(xs + n * 8u * x_line(MODE) + u * 64u + 32u);
                B = make_uint4(lo.x, lo.y, hi.x, hi.y);
            } else {
                B = lds128(xs + n * 8u * x_line(MODE) + u * 64u);
            }
            uint64_t f = 0ull, sum = 0ull;
            if constexpr (!UP) f = lds64x(fs + (u * MID_PAIRS + n * 8u) * 4u);
            if constexpr (affine(MODE)) sum = lds64x(fs + ((4u + u) * MID_PAIRS + n * 8u) * 4u);
#pragma unroll
            for (uint32_t t = 0; t < 2; t++) {
                const uint32_t i = 2u * t;
                float c[4], d[4];
                mma0(c, p[i][0], p[i + 1][0], p[i][1], p[i + 1][1], B.x, B.y);
                if constexpr (MODE == M_NV) mma0(d, p[i][2], p[i + 1][2], p[i][3], p[i + 1][3], B.z, B.w);
                else mma(c, p[i][2], p[i + 1][2], p[i][3], p[i + 1][3], B.z, B.w);
#pragma unroll
                for (uint32_t h = 0; h < 2; h++) {
                    uint64_t &to = acc[t][h][n];
                    const uint64_t c2 = pack2(c[2 * h], c[2 * h + 1]);
                    if constexpr (MODE == M_NV) {
                        const uint64_t d2 = pack2(d[2 * h], d[2 * h + 1]);
                        if constexpr (UP) to = fma2(s1[i + h], d2, fma2(s[i + h], c2, to));
                        else to = fma2(f, fma2(s1[i + h], d2, mul2(s[i + h], c2)), to);
                    } else {
                        to = fma2(s[i + h], UP ? c2 : mul2(f, c2), to);
                    }
                    if constexpr (affine(MODE)) to = fma2(b[i + h], sum, to);
                }
            }
        }
    }
}

// grid (blocks of 128 rows, tiles).
template <int MODE, bool UP>
__global__ void __launch_bounds__(MID_THREADS, ctas(MODE)) mid_product(const MidParams P) {
    constexpr uint32_t LINE = line(MODE), XL = x_line(MODE), STAGE = stage_bytes(MODE), RINGS = ring(MODE);
    constexpr uint32_t X_AT = MID_ROWS * LINE, F_AT = X_AT + MID_PAIRS * XL;
    static_assert(MID_PAIRS * HB * 4u <= RINGS * STAGE, "the epilogue's h takes the ring's room");
    extern __shared__ __align__(16) uint8_t sm[];
    ptx::griddep_wait();
    ptx::griddep_launch_dependents();
    if (blockIdx.y >= *P.tile_count) return;
    const uint32_t tid = threadIdx.x, warp = tid >> 5, lane = tid & 31u, r = lane >> 2, q = lane & 3u;
    // (plain loads: what the kernels before wrote, this one may have started beside them)
    const uint32_t e = P.tiles[2u * blockIdx.y], r0 = P.tiles[2u * blockIdx.y + 1u];
    const uint32_t place = P.offsets[e] + r0;
    const uint32_t np = tmin<uint32_t>(P.offsets[e + 1u] - place, MID_PAIRS), nt = (np + 7u) / 8u;
    const uint32_t nu = P.k / 32u, steps = (nu + 3u) / 4u, srow = scale_bytes(MODE, P.groups);

    // the lane's rows r, r + 8 of two tiles; UP: gate and up of 8 columns are a tile
    const uint32_t row0 = blockIdx.x * (UP ? HC : MID_ROWS) + warp * (UP ? 16u : 32u);
    const bool active = row0 < P.n;
    const size_t first = (size_t)e * (UP ? 2u : 1u) * P.n + (active ? row0 : 0u) + r;
    const size_t dr = UP ? P.n : 8u, dt = UP ? 8u : 16u;  // rows on to the lane's second, and to the next tile
    const uint8_t *const w0 = P.w + first * P.row_bytes, *const s0 = P.s + first * srow, *const b0 = P.a + first * srow;
    const uint32_t sm0 = ptx::smem_u32(sm);

    // half a warp copies a pair's values, a quad the factors and sums of a pair's four units
    constexpr uint32_t VI = MID_PAIRS / (2u * MID_WARPS), FI = (MID_PAIRS + 8u * MID_WARPS - 1u) / (8u * MID_WARPS);
    auto image = [&](uint32_t pr) {  // in units of 16 bytes
        const uint32_t at = place + (pr < np ? pr : 0u);
        return (UP ? P.sorted_pairs[at] / P.S : at) * (steps * (step_bytes(1) / 16u));
    };
    const uint32_t vp = 2u * warp + (lane >> 4), fp = 8u * warp + r;
    uint32_t vo[VI], fo[FI];
#pragma unroll
    for (uint32_t i = 0; i < VI; i++) vo[i] = image(vp + 2u * MID_WARPS * i) + (lane & 15u);
#pragma unroll
    for (uint32_t i = 0; i < FI; i++) fo[i] = image(fp + 8u * MID_WARPS * i) + 16u;
    const uint32_t vd = X_AT + vp * XL + (lane & 15u) * 16u, fd = F_AT + (q * MID_PAIRS + fp) * 4u;
    // 3-bit codes: the 16-byte blocks of memory that hold a step's 14 words
    const uint32_t rw = P.row_bytes / 4u, misplaced = MODE == M_CB3 ? r * rw : 0u;
    auto issue = [&](uint32_t j, uint32_t slot) {
        if (j < steps) {
            const uint32_t st = sm0 + slot * STAGE;
            if (active) {
#pragma unroll
                for (uint32_t i = 0; i < 4; i++) {
                    const uint8_t *g = w0 + ((i & 1u) * dr + (i >> 1) * dt) * P.row_bytes;
                    const uint32_t d = st + (warp * 32u + 8u * i + r) * LINE;
                    if constexpr (MODE == M_CB3) {
                        auto block = [&](uint32_t k) {
                            const Cb3Block c = cb3_block(misplaced, j, k, P.row_bytes);
                            ptx::cp_async_16(d + k * 16u, g + c.at, c.bytes);
                        };
                        block(q);
                        // 14 words from a block's fourth on: a fifth block
                        if (((misplaced + 128u * j / 10u) & 3u) == 3u && q == i) block(4u);
                    } else if constexpr (MODE == M_CB2) {
                        const uint32_t in = 4u * j + q < nu;
                        ptx::cp_async_8(d + q * 8u, g + (in ? (4u * j + q) * 8u : 0u), in ? 8u : 0u);
                    } else if constexpr (MODE == M_A6) {
#pragma unroll
                        for (uint32_t k = 0; k < 3; k++) {
                            const uint32_t o = (q + 4u * k) * 8u, in = 96u * j + o < P.row_bytes;
                            ptx::cp_async_8(d + o, g + (in ? 96u * j + o : 0u), in ? 8u : 0u);
                        }
                    } else {
                        constexpr uint32_t STEP = MODE == M_A8 ? 128u : 64u;
#pragma unroll
                        for (uint32_t k = 0; k < STEP / 64u; k++) {
                            const uint32_t o = (q + 4u * k) * 16u, in = STEP * j + o < P.row_bytes;
                            ptx::cp_async_16(d + o, g + (in ? STEP * j + o : 0u), in ? 16u : 0u);
                        }
                    }
                }
            }
            const uint8_t *const x = P.x + j * step_bytes(1);
#pragma unroll
            for (uint32_t i = 0; i < VI; i++)
                ptx::cp_async_16_if(vp + 2u * MID_WARPS * i < np, st + vd + 2u * MID_WARPS * i * XL,
                                    x + (size_t)vo[i] * 16u, 16u);
#pragma unroll
            for (uint32_t i = 0; i < FI; i++)
                if ((!UP || affine(MODE)) && fp + 8u * MID_WARPS * i < np) {
                    const uint8_t *const g = x + (size_t)fo[i] * 16u + q * 4u;
                    const uint32_t d = st + fd + 32u * MID_WARPS * i;
                    if constexpr (!UP) ptx::cp_async_4(d, g, 4u);
                    if constexpr (affine(MODE)) ptx::cp_async_4(d + 16u * MID_PAIRS, g + 16u, 4u);
                }
        }
        ptx::cp_async_commit();
    };
    // scales of unit q of a step, a step ahead, in registers
    uint32_t raw[2], rawb[2] = {0u, 0u}, nraw[4], nrawb[4] = {0u, 0u, 0u, 0u};
    auto fetch = [&](uint32_t j) {
        const uint32_t o = scale_entry<MODE>(tmin<uint32_t>(4u * j + q, nu - 1u), P.gshift);
#pragma unroll
        for (uint32_t i = 0; i < 4; i++) {
            const size_t row = ((i & 1u) * dr + (i >> 1) * dt) * srow;
            nraw[i] = raw_scale<MODE>(s0 + row + o);
            if constexpr (affine(MODE)) nrawb[i] = raw_scale<MODE>(b0 + row + o);
        }
    };
    for (uint32_t i = 0; i + 1u < RINGS; i++) issue(i, i);
    fetch(0u);
    Table<MODE> tab;
    tab.load(P.a);

    uint64_t acc[2][2][MID_BLOCKS];
#pragma unroll
    for (uint32_t t = 0; t < 4; t++)
#pragma unroll
        for (uint32_t n = 0; n < MID_BLOCKS; n++) acc[t >> 1][t & 1][n] = 0ull;

    const uint32_t row = sm0 + (warp * 32u + r) * LINE, xs = sm0 + X_AT + r * XL + q * (MODE == M_NV ? 8u : 16u),
                   fs = sm0 + F_AT + q * 8u;
    uint32_t slot = 0;
    for (uint32_t j = 0; j < steps; j++) {
        wait_groups<(int)RINGS - 2>();
        __syncthreads();  // the step has landed, and the slot of the step before is free
        issue(j + RINGS - 1u, slot == 0u ? RINGS - 1u : slot - 1u);
#pragma unroll
        for (uint32_t t = 0; t < 2; t++) {
            raw[t] = nraw[2 * t] | nraw[2 * t + 1] << 16;
            if constexpr (affine(MODE)) rawb[t] = nrawb[2 * t] | nrawb[2 * t + 1] << 16;
        }
        if (j + 1u < steps) fetch(j + 1u);
        if (active) {
            const uint32_t on = slot * STAGE;
            const uint32_t c0 = MODE == M_CB3 ? 128u * j % 10u : 0u, o = MODE == M_CB3 ? (misplaced + 128u * j / 10u) % 4u * 4u : 0u;
            switch (nt) {
                case 1: mid_step<MODE, UP, 1>(row + on + o, xs + on, fs + on, c0, raw, rawb, tab, lane, acc); break;
                case 2: mid_step<MODE, UP, 2>(row + on + o, xs + on, fs + on, c0, raw, rawb, tab, lane, acc); break;
                default: mid_step<MODE, UP, 3>(row + on + o, xs + on, fs + on, c0, raw, rawb, tab, lane, acc);
            }
        }
        slot = slot + 1u == RINGS ? 0u : slot + 1u;
    }
    wait_groups<0>();

    const float s2 = MODE == M_NV ? __ldg((const float *)P.a + e) : affine(MODE) ? CODE_UNIT : 1.f;
    if constexpr (!UP) {
        if (!active) return;
        float *const z = (float *)P.out;
        float bias[4];
#pragma unroll
        for (uint32_t i = 0; i < 4; i++)
            bias[i] = load_bias(P.bias, P.bias_dtype, (size_t)e * P.n + row0 + 8u * i + r);
#pragma unroll
        for (uint32_t n = 0; n < MID_BLOCKS; n++)
#pragma unroll
            for (uint32_t k = 0; k < 2; k++) {
                const uint32_t pr = 8u * n + 2u * q + k;
                if (pr < np) {
                    const uint32_t pair = P.sorted_pairs[place + pr];
                    const float wt = __ldg(P.weights + pair);
                    float *const to = z + (size_t)pair * P.n + row0 + r;
#pragma unroll
                    for (uint32_t i = 0; i < 4; i++) {
                        const float2 v = unpack2(acc[i >> 1][i & 1][n]);
                        to[8u * i] = fmaf(k ? v.y : v.x, s2 * wt, bias[i] * wt);
                    }
                }
            }
    } else {
        __syncthreads();  // every warp has left the ring
        float *const hb = (float *)sm;
        if (active) {
            float tf[MID_BLOCKS][2];
#pragma unroll
            for (uint32_t n = 0; n < 2 * MID_BLOCKS; n++) {
                const uint32_t pr = 4u * (n & ~1u) + 2u * q + (n & 1u);
                tf[n >> 1][n & 1] = pr < np ? P.factor[P.sorted_pairs[place + pr] / P.S] : 0.f;
            }
#pragma unroll
            for (uint32_t t = 0; t < 2; t++) {
                const uint32_t c = warp * 16u + 8u * t + r;
                const size_t bo = (size_t)e * 2u * P.n + row0 + 8u * t + r;
                const float bg = load_bias(P.bias, P.bias_dtype, bo), bu = load_bias(P.bias, P.bias_dtype, bo + P.n);
#pragma unroll
                for (uint32_t n = 0; n < MID_BLOCKS; n++) {
                    const float2 g = unpack2(acc[t][0][n]), u = unpack2(acc[t][1][n]);
                    const uint32_t pr = 8u * n + 2u * q;
                    if (pr < np) hb[pr * HB + c] = glu_act(P.act, fmaf(g.x * s2, tf[n][0], bg)) * fmaf(u.x * s2, tf[n][0], bu);
                    if (pr + 1u < np)
                        hb[(pr + 1u) * HB + c] = glu_act(P.act, fmaf(g.y * s2, tf[n][1], bg)) * fmaf(u.y * s2, tf[n][1], bu);
                }
            }
        }
        __syncthreads();
        // a warp writes a unit of 32 columns of a pair; the row of CTAs all of the last step's
        constexpr uint32_t HU = HC / 32u;
        const uint32_t u0 = blockIdx.x * HU, units = P.n / 32u, hsteps = (units + 3u) / 4u;
        const uint32_t end = blockIdx.x + 1u == gridDim.x ? 4u * hsteps : u0 + HU;
        for (uint32_t o = warp; o < (end - u0) * np; o += MID_WARPS) {
            const uint32_t pr = o / (end - u0), un = u0 + o % (end - u0);
            const float h = un < units ? hb[pr * HB + (un - u0) * 32u + lane] : 0.f;  // zeros past the last column
            float scale, factor;
            unit_scale(__reduce_max_sync(FULL, __float_as_uint(h) & 0x7FFFFFFFu), scale, factor);
            const bool part = P.order == 1 && (lane & 1u);  // a sixteenth, meets a 16-fold pair
            const __half b = __float2half_rn(part ? h * scale * 0.0625f : h * scale);
            // The sum that meets the affine biases is that of the rounded values, which the codes
            // meet: a rounding then counts with the weight c s + b, not with c s, which is many
            // times that in a group whose codes lie close together.
            float sum = __half2float(b) * (part ? 16.f / CODE_UNIT : 1.f / CODE_UNIT);
            if (P.sums)
#pragma unroll
                for (int d = 16; d > 0; d >>= 1) sum += __shfl_xor_sync(FULL, sum, d);
            uint8_t *img = (uint8_t *)P.out + ((size_t)(place + pr) * hsteps + (un >> 2)) * step_bytes(1);
            ((uint16_t *)(img + (un & 3u) * 64u))[b_place(P.order, lane)] = __half_as_ushort(b);
            if (lane == 0) {
                ((float *)(img + 256u))[un & 3u] = factor;
                ((float *)(img + 272u))[un & 3u] = sum * factor;
            }
        }
    }
}

constexpr uint32_t IMAGE_WARPS = 8;
constexpr uint32_t ROUTE_FEW = 4096;  // pairs up to which one CTA routes them

struct RouteParams {
    const uint32_t *ids;
    uint32_t *offsets, *sorted_pairs, *tiles, *tile_count, *err;
    uint32_t R, E;
};

// The pairs by expert and the tiles of each expert, by one CTA beside those that write the
// images (three launches less). A pair's column is computed by itself, so the order of an
// expert's pairs, which the atomics leave open, changes no result.
__device__ void route_few(const RouteParams &P) {
    __shared__ uint32_t at[ROUTE_MAX_E + 4], sums[IMAGE_WARPS];
    const uint32_t tid = threadIdx.x, lane = tid & 31u, warp = tid >> 5;
    constexpr uint32_t T = 32 * IMAGE_WARPS, EACH = ROUTE_MAX_E / T;
    for (uint32_t i = tid; i < ROUTE_MAX_E; i += T) at[i] = 0u;
    __syncthreads();
    for (uint32_t p = tid; p < P.R; p += T) {
        const uint32_t id = __ldg(P.ids + p);
        if (id < P.E) atomicAdd(&at[id], 1u);
        else atomicOr(P.err, ERR_BAD_ID);
    }
    __syncthreads();
    // pairs (at most 4,096) and tiles (at most 4,096 / 24 + 1,024) before each expert, in one word
    uint32_t n[EACH], own = 0u;
#pragma unroll
    for (uint32_t i = 0; i < EACH; i++) {
        n[i] = at[EACH * tid + i];
        own += n[i] | ((n[i] + MID_PAIRS - 1u) / MID_PAIRS) << 16;
    }
    uint32_t sum = own;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const uint32_t o = __shfl_up_sync(FULL, sum, d);
        if (lane >= (uint32_t)d) sum += o;
    }
    if (lane == 31u) sums[warp] = sum;
    __syncthreads();
    sum -= own;
    for (uint32_t w = 0; w < warp; w++) sum += sums[w];
#pragma unroll
    for (uint32_t i = 0; i < EACH; i++) {
        const uint32_t e = EACH * tid + i;
        at[e] = sum & 0xFFFFu;
        if (e <= P.E) P.offsets[e] = sum & 0xFFFFu;
        for (uint32_t r0 = 0, t = sum >> 16; r0 < n[i]; r0 += MID_PAIRS, t++) {
            P.tiles[2u * t] = e;
            P.tiles[2u * t + 1u] = r0;
        }
        sum += n[i] | ((n[i] + MID_PAIRS - 1u) / MID_PAIRS) << 16;
    }
    if (tid == T - 1u) {
        *P.tile_count = sum >> 16;
        if (P.E == ROUTE_MAX_E) P.offsets[P.E] = sum & 0xFFFFu;
    }
    __syncthreads();
    for (uint32_t p = tid; p < P.R; p += T) {
        const uint32_t id = __ldg(P.ids + p);
        if (id < P.E) P.sorted_pairs[atomicAdd(&at[id], 1u)] = p;
    }
}

// The tokens' images, in the order of MODE's codes, and the power of two of each. A CTA a
// token: the largest |value| first, so that the products need no factor for each unit.
// With up to ROUTE_FEW pairs one more CTA routes them.
template <int MODE>
__global__ void __launch_bounds__(32 * IMAGE_WARPS) mid_images(const void *x, int dt, uint32_t m, uint32_t k, uint8_t *img,
                                                               float *tf, const RouteParams route) {
    ptx::griddep_launch_dependents();
    if (blockIdx.x == m) {
        route_few(route);
        return;
    }
    __shared__ uint32_t most[IMAGE_WARPS];
    const uint32_t lane = threadIdx.x & 31u, warp = threadIdx.x >> 5, steps = (k + 127u) / 128u;
    const size_t row = (size_t)blockIdx.x * k;
    uint32_t mb = 0u;
    for (uint32_t c = 4u * threadIdx.x; c < k; c += 128u * IMAGE_WARPS) {
        const uint32_t M = 0x7FFFFFFFu;
        const float4 v = load_x4(x, dt, row + c);
        mb = max(mb, max(max(__float_as_uint(v.x) & M, __float_as_uint(v.y) & M),
                         max(__float_as_uint(v.z) & M, __float_as_uint(v.w) & M)));
    }
    mb = __reduce_max_sync(FULL, mb);
    if (lane == 0) most[warp] = mb;
    __syncthreads();
    mb = __reduce_max_sync(FULL, most[lane % IMAGE_WARPS]);
    float scale, factor;
    unit_scale(mb, scale, factor);
    if (threadIdx.x == 0) tf[blockIdx.x] = factor;
    for (uint32_t j = warp; j < steps; j += IMAGE_WARPS) {
        const uint32_t c = j * 128u + 4u * lane;
        float4 v = c < k ? load_x4(x, dt, row + c) : make_float4(0.f, 0.f, 0.f, 0.f);
        uint8_t *const to = img + ((size_t)blockIdx.x * steps + j) * step_bytes(1);
        if constexpr (affine(MODE)) {
            float sum = (v.x * scale + v.y * scale) + (v.z * scale + v.w * scale);
#pragma unroll
            for (int d = 1; d < 8; d <<= 1) sum += __shfl_xor_sync(FULL, sum, d);
            if ((lane & 7u) == 0u) ((float *)(to + 272u))[lane >> 3] = sum * (1.f / CODE_UNIT);
        }
        v = in_order<MODE, 1>(v, scale, lane);
        ((uint2 *)to)[lane] = make_uint2(to_f16x2(v.x, v.y), to_f16x2(v.z, v.w));
    }
}

template <int MODE, bool UP>
cudaError_t product(const MidParams &P, uint32_t max_tiles, cudaStream_t st) {
    auto kern = mid_product<MODE, UP>;
    const size_t smem = (size_t)ring(MODE) * stage_bytes(MODE);
    static SmemSet smem_set;
    const cudaError_t e = ensure_dyn_smem(kern, smem, smem_set);
    if (e != cudaSuccess) return e;
    // a programmatic dependent of the kernel before it, which saves the launch's latency
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((P.n * (UP ? 2u : 1u) + MID_ROWS - 1u) / MID_ROWS, max_tiles);
    cfg.blockDim = dim3(MID_THREADS);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, P);
}

template <bool UP>
cudaError_t product_m(const MidParams &P, int mode, uint32_t max_tiles, cudaStream_t st) {
    switch (mode) {
        case M_A4:
        case M_A4U: return product<M_A4U, UP>(P, max_tiles, st);
        case M_A6: return product<M_A6, UP>(P, max_tiles, st);
        case M_A8: return product<M_A8, UP>(P, max_tiles, st);
        case M_NV: return product<M_NV, UP>(P, max_tiles, st);
        case M_MX: return product<M_MX, UP>(P, max_tiles, st);
        case M_CB2: return product<M_CB2, UP>(P, max_tiles, st);
        case M_CB3: return product<M_CB3, UP>(P, max_tiles, st);
        default: return product<M_CB4, UP>(P, max_tiles, st);
    }
}

inline uint64_t al256(uint64_t v) { return (v + 255u) & ~255ull; }
uint64_t images(uint64_t rows, uint32_t k) { return al256(rows * ((k + 127ull) / 128ull) * step_bytes(1)); }
uint32_t tiles_of(uint64_t R, uint32_t E) { return (uint32_t)(R / MID_PAIRS) + E + 1u; }

}  // namespace

// Up to MOE_MLP_MID_PAIRS pairs an expert, 24 with 6-bit codes. Measured against the grouped
// products with 128 experts of 2,816 x 704, us: 24 pairs an expert 329 / 559 (affine 4 bits),
// 299 / 395 (NVFP4), 419 / 579 (3-bit codebook), 477 / 566 (6 bits); 32 pairs 414 / 568, 378 / 404,
// 534 / 590, 605 / 577. The other formats were not measured beyond 16 pairs an expert (MXFP4 there
// 236 / 829 us, so its crossing lies higher) and take the same limit.
static uint64_t mid_limit(uint32_t E) { return tmin<uint64_t>((uint64_t)MOE_MLP_MID_PAIRS * E, 1u << 20); }

uint64_t mlp_mid_workspace(uint32_t m, uint32_t hidden, uint32_t inter, uint32_t S, uint32_t E) {
    // with more pairs than it takes, what fewer pairs in the same workspace need
    const uint64_t R = tmin<uint64_t>((uint64_t)m * S, mid_limit(E)), tokens = tmin<uint64_t>(m, R);
    return al256(8ull * tiles_of(R, E)) + images(tokens, hidden) + images(R, inter) + al256(4ull * tokens) + R * hidden * 4ull;
}

bool mlp_mid_supported(const MlpArgs &a) {
    const uint64_t R = (uint64_t)a.m * a.S;
    const int m1 = mode_of(*a.gate_up, a.hidden), m2 = mode_of(*a.down, a.inter);
    // (images are addressed by 32 bits in steps of 16 bytes)
    return R <= mid_limit(a.E) && R * ((tmax(a.hidden, a.inter) + 127ull) / 128u) * (step_bytes(1) / 16u) < 1ull << 32 && a.E <= MOE_ROUTE_MAX_EXPERTS && a.x_dtype != DT_F32 && a.out_dtype != DT_F32 &&
           m1 >= 0 && m2 >= 0 && (R <= 24ull * a.E || (m1 != M_A6 && m2 != M_A6)) && ((uintptr_t)a.x & 7u) == 0;
}

cudaError_t launch_mlp_mid(const MlpArgs &a, uint8_t *ws, uint8_t *own, cudaStream_t st) {
    const uint32_t R = a.m * a.S, max_tiles = tiles_of(R, a.E);
    WsLayout L;
    if (!ws_layout(R, a.E, &L)) return cudaErrorInvalidValue;
    uint32_t *const err = (uint32_t *)(ws + L.err), *const tc = (uint32_t *)(ws + L.tile_count);
    uint32_t *const offsets = (uint32_t *)(ws + L.offsets);
    uint32_t *const sp = (uint32_t *)(ws + L.sorted_pairs), *const tiles = (uint32_t *)own;
    uint8_t *const xi = own + al256(8ull * max_tiles), *const hi = xi + images(a.m, a.hidden);
    float *const tf = (float *)(hi + images(R, a.inter)), *const z = tf + al256(4ull * a.m) / 4u;
    cudaError_t e = cudaSuccess;
    const bool one = R <= ROUTE_FEW;
    if (!one)
        e = launch_route(a.ids, R, a.E, MID_PAIRS, (uint32_t *)(ws + L.counts), offsets, sp, tiles, tc, max_tiles,
                         (uint32_t *)(ws + L.chunk_hist), (uint32_t *)(ws + L.chunk_base), L.chunks, err, nullptr, 0, 0, st);
    if (e != cudaSuccess) return e;
    const int m1 = mode_of(*a.gate_up, a.hidden), m2 = mode_of(*a.down, a.inter);
    auto images_of = order_of(m1) == 1 ? mid_images<M_A4> : order_of(m1) == 2 ? mid_images<M_A8>
                   : m1 == M_A6 ? mid_images<M_A6> : mid_images<M_NV>;
    images_of<<<a.m + (one ? 1u : 0u), 32 * IMAGE_WARPS, 0, st>>>(a.x, a.x_dtype, a.m, a.hidden, xi, tf,
                                                                  RouteParams{a.ids, offsets, sp, tiles, tc, err, R, a.E});
    if ((e = cudaGetLastError()) != cudaSuccess) return e;

    MidParams P{};
    P.w = (const uint8_t *)a.gate_up->packed; P.s = (const uint8_t *)a.gate_up->scales;
    P.a = (const uint8_t *)a.gate_up->aux; P.bias = a.gate_up->bias; P.bias_dtype = (int)a.gate_up->bias_dtype;
    P.x = xi; P.factor = tf; P.out = hi;
    P.offsets = offsets; P.sorted_pairs = sp; P.tiles = tiles; P.tile_count = tc;
    P.k = a.hidden; P.n = a.inter; P.S = a.S;
    P.row_bytes = (uint32_t)moe_packed_row_bytes(a.gate_up->fmt, a.gate_up->bits, a.hidden);
    P.groups = a.hidden / a.gate_up->group_size; P.gshift = log2_units(*a.gate_up);
    P.act = a.act; P.order = order_of(m2); P.sums = affine(m2);
    e = product_m<true>(P, m1, max_tiles, st);
    if (e != cudaSuccess) return e;
    P.w = (const uint8_t *)a.down->packed; P.s = (const uint8_t *)a.down->scales;
    P.a = (const uint8_t *)a.down->aux; P.bias = a.down->bias; P.bias_dtype = (int)a.down->bias_dtype;
    P.x = hi; P.out = z; P.weights = a.weights;
    P.k = a.inter; P.n = a.hidden;
    P.row_bytes = (uint32_t)moe_packed_row_bytes(a.down->fmt, a.down->bits, a.inter);
    P.groups = a.inter / a.down->group_size; P.gshift = log2_units(*a.down);
    e = product_m<false>(P, m2, max_tiles, st);
    if (e != cudaSuccess) return e;
    return launch_combine(z, nullptr, a.ids, a.residual, a.out, a.m, a.S, a.hidden, a.E, DT_F32, a.out_dtype, st);
}

}  // namespace moe
