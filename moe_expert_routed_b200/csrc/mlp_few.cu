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
// plane holds bf16 x exactly down to 2^-31 of the unit's largest value and f16 x down to
// 2^-28 (2^-27 and 2^-24 where x meets 16-fold codes); f32 x takes two, 22 bits. h, the f32 result of mlp_up, takes one for a bf16 result (11
// bits, 3 more than the rounding to bf16 that the result gets anyway) and two otherwise.
//   Scales of weights and of x are applied to f32 sums of one unit. The four lanes
// that share a row each hold another unit (their 16-byte load), so a column belongs to
// one unit: lane q's x stands in column q, the other lanes are zero there, and the
// accumulator keeps the four units apart in four columns; the eight columns hold two
// sets (two pairs, or the two planes of one pair).
// tcgen05's 128-row tiles with one or two columns in use would waste more than this
// does, and need their operand in shared or tensor memory.
//   Measured, 128 experts of 2,816 x 704, top-8, affine 4 bits: 1 token 14.6 us (floor 4.1),
// 8 tokens 58 us (26.4; the grouped products 270); NVFP4, 4,096 x 768, 5 tokens 61 us (28.7).
// Neither memory (39 and 24 % busy at 8 tokens) nor a pipe is full: the prologues take 11.7 us
// of mlp_up's 35.8 and 9.3 of mlp_down's 28.5, the rest issues in half of its cycles. Three
// CTAs an SM 65 us, two ring stages the same, one unit of columns a CTA 69, the down weights
// prefetched into L2 67. Without the dependent launch one token takes 17.9 us.
#include "common.cuh"
#include "internal.h"
#include "mlp_codes.cuh"
#include "ptx.cuh"

namespace moe {
namespace {

constexpr uint32_t FEW_THREADS = 256, FEW_WARPS = 8;
constexpr uint32_t FEW_MAX_R = MOE_MLP_FEW_PAIRS;
constexpr uint32_t ID_LOOPS = FEW_MAX_R / FEW_THREADS;  // a thread's in the prologues
constexpr uint32_t FEW_MAX_TOKENS = MOE_MLP_FEW_TOKENS;  // rows of mlp_down's per-warp sums
constexpr uint32_t RING = 3;             // steps of a warp in flight
constexpr uint32_t UP_TILES = 2;         // mlp_up: tiles of 16 rows a warp works on at once
constexpr uint32_t UP_PARTS = 4;         // mlp_up: warps that share a pair of tiles, each a part of hidden
constexpr uint32_t MAX_SPLIT = 4;        // mlp_down: CTAs that share 16 columns
constexpr uint32_t FEW_ALONE_R = 16;     // pairs up to which mlp_down's CTAs share no columns
constexpr uint32_t SMS = 148;
constexpr size_t FEW_SMEM = 216 * 1024;

// Planes of x by its type, of h by the result's.
constexpr int x_planes(int dt) { return dt == DT_F32 ? 2 : 1; }
__host__ __device__ constexpr int h_planes(int out_dtype) { return out_dtype == DT_BF16 ? 1 : 2; }

// ------------------------------------------------------------------ one step

// Where a lane reads its part of the step images (shared addresses): for each block of
// columns the B registers, with `move` all ones where they move with the step, and the
// factors and sums of its accumulator columns. The lanes whose k are not their column's
// unit read zeros. Pairs past a pass's last are not masked: their columns hold what the
// memory holds, mix with no other column and are dropped.
template <int NB>
struct StepAt {
    uint32_t b[NB], f[NB], move;
};

template <int PLANES, int NB>
__device__ __forceinline__ StepAt<NB> step_at(uint32_t base, uint32_t stride, uint32_t zeros, uint32_t lane) {
    StepAt<NB> A;
    const uint32_t q = lane & 3u;
    const bool active = ((lane >> 2) & 3u) == q;  // this lane's k of column lane / 4 are that column's unit
    A.move = active ? FULL : 0u;
#pragma unroll
    for (uint32_t n = 0; n < NB; n++) {
        const uint32_t set = 2u * n + (lane >> 4), pair = set / PLANES, plane = set % PLANES;
        A.b[n] = active ? base + pair * stride + plane * 256u + q * 64u : zeros;
        // accumulator columns 2q, 2q + 1: units 2 (q mod 2) and the next of set 2n + q / 2
        A.f[n] = base + (2u * n + (q >> 1)) / PLANES * stride + PLANES * 256u + (q & 1u) * 16u;
    }
    return A;
}

// Scales (and affine biases) that a lane applies: of rows r and r + 8 and the two units of
// its accumulator columns; NVFP4 units have two.
template <int MODE>
struct Scales {
    static constexpr int PARTS = MODE == M_NV ? 2 : 1, UNITS = MODE == M_A4 ? 1 : 2;
    float s[PARTS][2][UNITS];  // [part of a unit][row][unit]
    float b[2][UNITS];
};

// a: shared address of row r's scales, to8: bytes to row r + 8, tob: to the biases; i, d:
// bytes to the first unit's entry and on to the second's.
template <int MODE, bool CENTRED>
__device__ __forceinline__ void load_scales(Scales<MODE> &S, uint32_t a, uint32_t to8, uint32_t tob, uint32_t i,
                                            uint32_t d) {
#pragma unroll
    for (int h = 0; h < 2; h++) {
#pragma unroll
        for (int u = 0; u < Scales<MODE>::UNITS; u++) {
            const uint32_t at = a + i + (u ? d : 0u) + (h ? to8 : 0u);
            if constexpr (affine(MODE)) {
                S.s[0][h][u] = bf16_bits_to_f32(lds16(at));
                S.b[h][u] = bf16_bits_to_f32(lds16(at + tob));
                if constexpr (CENTRED) S.b[h][u] = fmaf(middle(MODE), S.s[0][h][u], S.b[h][u]);
            } else if constexpr (codebook(MODE)) {
                S.s[0][h][u] = f16_bits_to_f32(lds16(at));
            } else if constexpr (MODE == M_MX) {
                S.s[0][h][u] = e8m0_to_f32(lds8(at));
            } else {
                from_e4m3x2(lds16(at), S.s[0][h][u], S.s[Scales<MODE>::PARTS - 1][h][u]);
            }
        }
    }
}

// 16 rows x 4 units: wa, wb the lane's unit of rows r and r + 8.
template <int MODE, bool CENTRED, int NB>
__device__ __forceinline__ void tile_step(const uint32_t (&wa)[words(MODE)], const uint32_t (&wb)[words(MODE)],
                                          const Table<MODE> &T, const uint32_t (&B)[NB][16], const float (&f)[NB][2],
                                          const float (&xs)[NB][2], const Scales<MODE> &C, float (&acc)[NB][2]) {
    constexpr int PARTS = Scales<MODE>::PARTS, QPP = 4 / PARTS;  // quarters of a unit in a part
#pragma unroll
    for (int h = 0; h < PARTS; h++) {
        float c[NB][4];
#pragma unroll
        for (int i = 0; i < QPP; i++) {
            const int t = h * QPP + i;
            uint32_t pa[4], pb[4];
            expand<MODE, CENTRED>(wa, t, T, pa);
            expand<MODE, CENTRED>(wb, t, T, pb);
#pragma unroll
            for (int n = 0; n < NB; n++) {
                if (i == 0) mma0(c[n], pa[0], pb[0], pa[1], pb[1], B[n][4 * t], B[n][4 * t + 1]);
                else mma(c[n], pa[0], pb[0], pa[1], pb[1], B[n][4 * t], B[n][4 * t + 1]);
                mma(c[n], pa[2], pb[2], pa[3], pb[3], B[n][4 * t + 2], B[n][4 * t + 3]);
            }
        }
#pragma unroll
        for (int n = 0; n < NB; n++)
#pragma unroll
            for (int k = 0; k < 2; k++) {
                const float c0 = c[n][2 * k], c1 = c[n][2 * k + 1];
                if constexpr (MODE == M_A4)
                    acc[n][k] = fmaf(C.s[0][k][0], fmaf(c0, f[n][0], c1 * f[n][1]), acc[n][k]);
                else
                    acc[n][k] = fmaf(C.s[h][k][0], c0 * f[n][0],
                                     fmaf(C.s[h][k][Scales<MODE>::UNITS - 1], c1 * f[n][1], acc[n][k]));
            }
    }
    if constexpr (MODE == M_A4) {
#pragma unroll
        for (int n = 0; n < NB; n++)
#pragma unroll
            for (int k = 0; k < 2; k++) acc[n][k] = fmaf(C.b[k][0], xs[n][0] + xs[n][1], acc[n][k]);
    } else if constexpr (affine(MODE)) {
#pragma unroll
        for (int n = 0; n < NB; n++)
#pragma unroll
            for (int k = 0; k < 2; k++)
                acc[n][k] = fmaf(C.b[k][0], xs[n][0], fmaf(C.b[k][1], xs[n][1], acc[n][k]));
    }
}

// One step of T tiles: st the stage's address for this lane (+ lane pieces), sc that of row r's
// scales of the first tile (tot bytes on to the next tile's), `on` bytes past at the images.
template <int MODE, int PLANES, int NB, int T>
__device__ __forceinline__ void step(uint32_t st, uint32_t sc, uint32_t tot, uint32_t to8, uint32_t tob, uint32_t i,
                                     uint32_t d, uint32_t word_codes, const Table<MODE> &tab, const StepAt<NB> &at,
                                     uint32_t on, uint32_t lane, float (&acc)[T][NB][2]) {
    uint32_t B[NB][16];
    float f[NB][2], xs[NB][2];
    const bool odd_plane = PLANES == 2 && (lane & 2u);
    constexpr bool CENTRED = centred(MODE, PLANES);
    const float plane = odd_plane ? 4.8828125e-4f : 1.f;  // 2^-11
    constexpr float unit = 1.f / code_unit(MODE, PLANES);
#pragma unroll
    for (int n = 0; n < NB; n++) {
#pragma unroll
        for (int k = 0; k < 4; k++) {
            const uint4 v = lds128(at.b[n] + (on & at.move) + 16u * k);
            B[n][4 * k] = v.x; B[n][4 * k + 1] = v.y; B[n][4 * k + 2] = v.z; B[n][4 * k + 3] = v.w;
        }
        const uint4 v = lds128(at.f[n] + on);
        f[n][0] = PLANES == 2 ? __uint_as_float(v.x) * plane : __uint_as_float(v.x);
        f[n][1] = PLANES == 2 ? __uint_as_float(v.z) * plane : __uint_as_float(v.z);
        xs[n][0] = odd_plane ? 0.f : __uint_as_float(v.y) * unit;  // the bias once a pair
        xs[n][1] = odd_plane ? 0.f : __uint_as_float(v.w) * unit;
    }
#pragma unroll
    for (uint32_t t = 0; t < T; t++) {
        uint32_t wa[words(MODE)], wb[words(MODE)];
        load_unit<MODE>(st + 2u * t * rows8(MODE), wa);
        load_unit<MODE>(st + (2u * t + 1u) * rows8(MODE), wb);
        join_words<MODE>(wa, word_codes);
        join_words<MODE>(wb, word_codes);
        Scales<MODE> C;
        load_scales<MODE, CENTRED>(C, sc + t * tot, to8, tob, i, d);
        tile_step<MODE, CENTRED, NB>(wa, wb, tab, B, f, xs, C, acc[t]);
    }
}

// Codes of a 3-bit word that come before unit u.
template <int MODE>
__device__ __forceinline__ uint32_t codes_before(uint32_t u) {
    return MODE == M_CB3 ? 32u * u % 10u : 0u;
}

// ------------------------------------------------------------------- routing

// The distinct valid experts of the pairs' ids (shared, past-the-last and invalid ones
// FULL) as bits, ascending ranks by prefix counts. All threads of the CTA call it;
// shared arrays of 32 and 33.
__device__ __forceinline__ uint32_t expert_mask(const uint32_t *ids, uint32_t *mask, uint32_t *base) {
    const uint32_t tid = threadIdx.x;
    if (tid < 32) mask[tid] = 0u;
    __syncthreads();
#pragma unroll
    for (uint32_t i = 0; i < ID_LOOPS; i++) {
        const uint32_t id = ids[tid + i * FEW_THREADS];
        if (id != FULL) atomicOr(&mask[id >> 5], 1u << (id & 31u));
    }
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
    uint8_t *hf;                     // h: [R][steps of inter][step_bytes(planes of h)]
    uint32_t *err;
    uint32_t m, R, S, E, H, I;       // H hidden, I inter
    uint32_t g1, g2, gshift1, gshift2;  // groups of a row; log2(units of 32 a group)
    int x_dtype, out_dtype, bias1_dtype, bias2_dtype, act;
    uint32_t rb1, rb2;               // bytes of a packed row
    int scale2_kind, down_order;     // 1: the down projection is NVFP4 (scale2 in a2); order of h's values
    uint32_t split, max_parts, slots;  // mlp_down: CTAs that share 16 columns, parts an expert, scale slots
    float *partial;                  // [split][m][H] sums of mlp_down's CTAs, where they share columns
    uint32_t *arrived;               // [H / 16], zeroed by mlp_up
};

// mlp_up. grid (blocks of units, pairs or experts). A CTA works for the expert of its
// pair, if no earlier pair has the same (or, with more pairs than experts, for its own
// expert), on units of 32 columns of h (units of mlp_down; 64 weight rows: tile t pairs gate rows 8t..8t+7 with up rows 8t..8t+7, so that a lane's two
// accumulator rows are the gate and the up of one column). Each pair of tiles has four
// warps, which take the steps of 128 codes in turn and run on into the CTA's next unit;
// x is written as step images once for all.
template <int MODE, int PLANES, int NB>
__global__ void __launch_bounds__(FEW_THREADS, NB <= 2 ? 2 : 1) mlp_up(const FewParams P) {
    constexpr uint32_t PP = 2 * NB / PLANES;  // pairs a pass
    constexpr uint32_t STAGE = UP_TILES * 2 * rows8(MODE), XSTEP = step_bytes(PLANES);
    extern __shared__ __align__(16) uint8_t sm[];
    __shared__ __align__(16) uint8_t zeros[64];
    __shared__ float red[UP_PARTS * PP * 64];  // [part][pair][gate / up][32 columns]
    __shared__ uint32_t wcount[ID_LOOPS * FEW_WARPS], pairs[FEW_MAX_R];

    const uint32_t tid = threadIdx.x, warp = tid >> 5, lane = tid & 31u;
    if (tid < 16) ((uint32_t *)zeros)[tid] = 0u;
    // mlp_down may start from here on: what came before this kernel is complete
    ptx::griddep_wait();
    ptx::griddep_launch_dependents();

    const bool by_pair = P.R <= P.E;
    const uint32_t e = by_pair ? __ldg(P.ids + blockIdx.y) : blockIdx.y;
    uint32_t id[ID_LOOPS];
#pragma unroll
    for (uint32_t i = 0; i < ID_LOOPS; i++) {
        const uint32_t p = tid + i * FEW_THREADS;
        id[i] = p < P.R ? __ldg(P.ids + p) : FULL;
    }
    if (blockIdx.x == 0 && blockIdx.y == 0) {
#pragma unroll
        for (uint32_t i = 0; i < ID_LOOPS; i++)
            if (tid + i * FEW_THREADS < P.R && id[i] >= P.E) atomicOr(P.err, ERR_BAD_ID);
        if (P.split > 1u)
            for (uint32_t i = tid; i < P.H / 16u; i += FEW_THREADS) P.arrived[i] = 0u;
    }
    if (e >= P.E) return;
    bool earlier = false;
    uint32_t mine_w[ID_LOOPS];
#pragma unroll
    for (uint32_t i = 0; i < ID_LOOPS; i++) {
        mine_w[i] = __ballot_sync(FULL, id[i] == e);
        if (lane == 0) wcount[i * FEW_WARPS + warp] = __popc(mine_w[i]);
        earlier |= by_pair && id[i] == e && tid + i * FEW_THREADS < blockIdx.y;
    }
    if (__syncthreads_or(earlier)) return;
    uint32_t np = 0;
#pragma unroll
    for (uint32_t i = 0; i < ID_LOOPS; i++) {
        uint32_t before = np;
#pragma unroll
        for (uint32_t k = 0; k < FEW_WARPS; k++) {
            const uint32_t n = wcount[i * FEW_WARPS + k];
            if (k < warp) before += n;
            np += n;
        }
        if (id[i] == e) pairs[before + __popc(mine_w[i] & ((1u << lane) - 1u))] = tid + i * FEW_THREADS;
    }
    if (np == 0u) return;

    const uint32_t r = lane >> 2, q = lane & 3u, tp = warp & 1u, part = warp >> 1;
    const uint32_t nu = P.H / 32u, steps = (nu + 3u) / 4u, units = P.I / 32u;
    const uint32_t row_bytes = P.rb1, srow = scale_bytes(MODE, P.g1), sblock = 32u * srow;
    uint8_t *const images = sm + FEW_WARPS * RING * STAGE;  // [pair][step]
    uint8_t *const scales = images + PP * steps * XSTEP;    // [2][gate, up scales, biases][32 rows]
    const uint32_t sm0 = ptx::smem_u32(sm), ring = sm0 + warp * RING * STAGE;
    const uint32_t sc0 = ptx::smem_u32(scales), sbytes = sblock * (affine(MODE) ? 4u : 2u);
    const size_t up = (size_t)P.I * row_bytes, next = 8u * (size_t)row_bytes;

    // requests of weights: unit, step, slot; the lane's row of the first tile
    const uint8_t *wrow = nullptr;
    uint32_t iu = 0, ij = 0, is = 0;
    auto issue = [&]() {
        if (iu < units) {
            const uint32_t in = 4u * ij + q < nu;  // past the row nothing is read, zeros are stored
            const uint8_t *g = wrow + (in ? unit_byte<MODE>(4u * ij + q) : 0u);
            const uint32_t st = ring + is + lane * piece(MODE);
            copy_unit<MODE>(st, g, in);
            copy_unit<MODE>(st + rows8(MODE), g + up, in);
            g += next;
            copy_unit<MODE>(st + 2u * rows8(MODE), g, in);
            copy_unit<MODE>(st + 3u * rows8(MODE), g + up, in);
            is = is + STAGE == RING * STAGE ? 0u : is + STAGE;
            ij += UP_PARTS;
            if (ij >= steps) {
                ij = part;
                iu += gridDim.x;
                wrow += (size_t)gridDim.x * 32u * row_bytes;
            }
        }
    };
    // a unit's scales (and affine biases): blocks of 32 contiguous rows, by the whole CTA
    auto issue_scales = [&](uint32_t unit, uint32_t buf) {
        if (unit >= units) return;
        const size_t g = ((size_t)e * 2u * P.I + unit * 32u) * srow, u = g + (size_t)P.I * srow;
        const uint32_t dst = sc0 + buf * sbytes;
        for (uint32_t o = tid * 16u; o < sblock; o += FEW_THREADS * 16u) {
            ptx::cp_async_16(dst + o, P.s1 + g + o, 16);
            ptx::cp_async_16(dst + sblock + o, P.s1 + u + o, 16);
            if constexpr (affine(MODE)) {
                ptx::cp_async_16(dst + 2u * sblock + o, P.a1 + g + o, 16);
                ptx::cp_async_16(dst + 3u * sblock + o, P.a1 + u + o, 16);
            }
        }
    };
    auto restart = [&]() {
        iu = part < steps ? blockIdx.x : units;
        ij = part;
        is = 0u;
        wrow = P.w1 + ((size_t)e * 2u * P.I + iu * 32u + 16u * tp + r) * row_bytes;
        issue_scales(blockIdx.x, 0u);
#pragma unroll
        for (uint32_t i = 0; i < RING; i++) {
            issue();
            ptx::cp_async_commit();
        }
    };
    restart();
    Table<MODE> tab;
    tab.load(P.a1);
    __syncthreads();  // pairs[]

    for (uint32_t pb = 0; pb < np; pb += PP) {
        const uint32_t npass = tmin<uint32_t>(PP, np - pb);
        if (pb) restart();
        for (uint32_t p = 0; p < npass; p++) {
            const size_t xrow = (size_t)(pairs[pb + p] / P.S) * P.H + 4u * lane;
#pragma unroll 4
            for (uint32_t j = warp; j < steps; j += FEW_WARPS) {
                const float4 v = j * 128u + 4u * lane < P.H ? load_x4(P.x, P.x_dtype, xrow + j * 128u)
                                                            : make_float4(0.f, 0.f, 0.f, 0.f);
                write_step<MODE, PLANES>(images + (p * steps + j) * XSTEP, v, lane);
            }
        }
        // what the epilogue of this warp's pair needs, requested now (a pass has at most 8)
        const bool mine = warp < npass;
        const uint32_t p_e = mine ? pairs[pb + warp] : 0u;
        float weight = 0.f;
        if (mine) {
            weight = __ldg(P.weights + p_e);
            if (P.scale2_kind) weight *= __ldg((const float *)P.a2 + e);
        }
        const float s2 = MODE == M_NV ? __ldg((const float *)P.a1 + e) : code_unit(MODE, PLANES);
        wait_groups<RING - 1>();  // the first unit's scales came with the first step
        __syncthreads();          // images, scales

        const StepAt<NB> at =
            step_at<PLANES, NB>(ptx::smem_u32(images) + part * XSTEP, steps * XSTEP, ptx::smem_u32(zeros), lane);
        uint32_t slot = 0, buf = 0;
        for (uint32_t unit = blockIdx.x; unit < units; unit += gridDim.x, buf ^= 1u) {
            float acc[UP_TILES][NB][2];
#pragma unroll
            for (uint32_t t = 0; t < UP_TILES; t++)
#pragma unroll
                for (int n = 0; n < NB; n++) acc[t][n][0] = acc[t][n][1] = 0.f;
            uint32_t on = 0;
            const uint32_t sc = sc0 + buf * sbytes + (16u * tp + r) * srow;
            issue_scales(unit + gridDim.x, buf ^ 1u);  // with this unit's first step
            for (uint32_t j = part; j < steps; j += UP_PARTS) {
                wait_groups<RING - 1>();
                const uint32_t u0 = tmin<uint32_t>(4u * j + 2u * (q & 1u), nu - 1u), u1 = tmin<uint32_t>(u0 + 1u, nu - 1u);
                const uint32_t i = scale_entry<MODE>(u0, P.gshift1);
                step<MODE, PLANES, NB, UP_TILES>(ring + slot + lane * piece(MODE), sc, 8u * srow, sblock, 2u * sblock, i,
                                                 scale_entry<MODE>(u1, P.gshift1) - i, codes_before<MODE>(4u * j + q),
                                                 tab, at, on, lane, acc);
                on += UP_PARTS * XSTEP;
                slot = slot + STAGE == RING * STAGE ? 0u : slot + STAGE;
                issue();
                ptx::cp_async_commit();
            }
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
                            red[((part * PP + p) * 2u + h) * 32u + 16u * tp + 8u * t + r] = v;
                        }
                    }
            // the next unit's scales: RING groups or more came after theirs, or wait for all
            if (steps >= RING * UP_PARTS) wait_groups<RING - 1>();
            else asm volatile("cp.async.commit_group;\n\tcp.async.wait_all;" ::: "memory");
            __syncthreads();
            if (mine) {  // one warp a pair: lane = column of h
                float g = 0.f, v = 0.f;
#pragma unroll
                for (uint32_t k = 0; k < UP_PARTS; k++) {
                    g += red[((k * PP + warp) * 2u) * 32u + lane];
                    v += red[((k * PP + warp) * 2u + 1u) * 32u + lane];
                }
                const size_t bo = (size_t)e * 2u * P.I + unit * 32u + lane;
                g = g * s2 + load_bias(P.bias1, P.bias1_dtype, bo);
                v = v * s2 + load_bias(P.bias1, P.bias1_dtype, bo + P.I);
                float h = glu_act(P.act, g) * v * weight;
                // this unit of the pair's step image
                const int planes = h_planes(P.out_dtype);
                const uint32_t un = unit & 3u;
                uint8_t *img = P.hf + ((size_t)p_e * ((units + 3u) / 4u) + (unit >> 2)) * step_bytes(planes);
                float scale, factor;
                unit_scale(__reduce_max_sync(FULL, __float_as_uint(h) & 0x7FFFFFFFu), scale, factor);
                const bool part = P.down_order == 1 && planes == 1 && (lane & 1u);  // a sixteenth, meets a 16-fold pair
                h *= part ? scale * 0.0625f : scale;
                uint16_t *dst = (uint16_t *)(img + un * 64u) + b_place(P.down_order, lane);
                // The sum that meets the affine biases is that of the rounded values, which the
                // codes meet: a rounding then counts with the weight c s + b, not with c s, which
                // is many times that in a group whose codes lie close together.
                float sum = 0.f, plane = part ? factor * 16.f : factor;
                for (int k = 0; k < planes; k++, dst += 128, plane *= 4.8828125e-4f) {  // 2^-11
                    const __half b = __float2half_rn(h);
                    *dst = __half_as_ushort(b);
                    sum = fmaf(__half2float(b), plane, sum);
                    h = (h - __half2float(b)) * 2048.f;
                }
#pragma unroll
                for (int d = 16; d > 0; d >>= 1) sum += __shfl_xor_sync(FULL, sum, d);
                float2 *fs = (float2 *)(img + planes * 256);
                if (lane == 0) fs[un] = make_float2(factor, sum);
                // units past inter in the last step are zero
                if (unit + 1u == units)
                    for (uint32_t z = un + 1u; z < 4u; z++) {
                        for (int k = 0; k < planes; k++) ((uint16_t *)(img + k * 256 + z * 64u))[lane] = 0;
                        if (lane == 0) fs[z] = make_float2(0.f, 0.f);
                    }
            }
            __syncthreads();  // red is read before the next unit's sums land there
        }
        asm volatile("cp.async.wait_all;" ::: "memory");
        if (pb + PP < np) __syncthreads();  // the images are read
    }
}

// mlp_down. grid (hidden / (16 T), split): a CTA holds T tiles, 16 T columns of out, and
// `split` CTAs share them. Their warps share the work items, (expert, part of its steps); each keeps sums of
// its own for every token, added in warp order, and with a split the last CTA to arrive
// adds the CTAs' sums in their order: no float atomics, one order. Weights and scales do
// not depend on mlp_up, so the ring's first steps are requested before waiting for it.
template <int MODE, int NPL, int NB, int T>
__global__ void __launch_bounds__(FEW_THREADS, NB <= 2 ? 2 : 1) mlp_down(const FewParams P) {
    constexpr uint32_t PP = 2 * NB / NPL, C = 16 * T;  // pairs a pass, columns
    constexpr uint32_t HSTEP = step_bytes(NPL), HAT = T * 2 * rows8(MODE), STAGE = HAT + PP * HSTEP;
    extern __shared__ __align__(16) uint8_t sm[];
    __shared__ __align__(16) uint8_t zeros[64];
    __shared__ uint32_t mask[32], base[33], ids_s[FEW_MAX_R], first[FEW_MAX_R + 1], pairs[FEW_MAX_R],
        experts[FEW_MAX_R], last_s;

    const uint32_t tid = threadIdx.x, warp = tid >> 5, lane = tid & 31u;
    if (tid < 16) ((uint32_t *)zeros)[tid] = 0u;
#pragma unroll
    for (uint32_t i = 0; i < ID_LOOPS; i++) {
        const uint32_t p = tid + i * FEW_THREADS;
        const uint32_t id = p < P.R ? __ldg(P.ids + p) : FULL;  // complete before mlp_up began
        ids_s[p] = id < P.E ? id : FULL;
        first[p] = 0u;
    }
    if (tid == 0) first[FEW_MAX_R] = 0u;
    __syncthreads();
    const uint32_t D = expert_mask(ids_s, mask, base);
    const uint32_t srow = scale_bytes(MODE, P.g2), sslot = C * srow * (affine(MODE) ? 2u : 1u);
    const uint32_t warp_bytes = RING * STAGE + P.slots * sslot;
    float *const ysm = (float *)(sm + FEW_WARPS * warp_bytes);  // [warp][token][C]
    for (uint32_t o = tid; o < FEW_WARPS * P.m * C; o += FEW_THREADS) ysm[o] = 0.f;
    __syncthreads();
    if (warp == 0) {
        // the pairs by expert, in their order: ranks, counts, firsts, places
        auto rank_of = [&](uint32_t id) { return base[id >> 5] + __popc(mask[id >> 5] & ((1u << (id & 31u)) - 1u)); };
        for (uint32_t o = 0; o < P.R; o += 32) {
            const uint32_t id = ids_s[o + lane], same = __match_any_sync(FULL, id);
            if (id != FULL && (same & ((1u << lane) - 1u)) == 0u) {
                const uint32_t x = rank_of(id);
                first[x + 1u] += __popc(same);
                experts[x] = id;
            }
            __syncwarp();
        }
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
        __syncwarp();
        for (uint32_t o = 0; o < P.R; o += 32) {  // first[x] runs to the next expert's and is put back below
            const uint32_t id = ids_s[o + lane], same = __match_any_sync(FULL, id), before = same & ((1u << lane) - 1u);
            const uint32_t x = id != FULL ? rank_of(id) : 0u;
            if (id != FULL) pairs[first[x] + __popc(before)] = (o + lane) | ((o + lane) / P.S) << 16;  // pair, token
            __syncwarp();
            if (id != FULL && before == 0u) first[x] += __popc(same);
            __syncwarp();
        }
        for (uint32_t o = (D + 31u) & ~31u; o > 0u; o -= 32) {  // from the top: first[x] = old first[x - 1]'s end
            const uint32_t x = o - 32u + lane;
            const uint32_t v = x < D && x > 0u ? first[x - 1u] : 0u;
            __syncwarp();
            if (x < D) first[x] = v;
            __syncwarp();
        }
    }
    __syncthreads();

    const uint32_t r = lane >> 2, q = lane & 3u;
    const uint32_t nu = P.I / 32u, steps = (nu + 3u) / 4u, row_bytes = P.rb2;
    const uint32_t row0 = blockIdx.x * C, warps = P.split * FEW_WARPS;
    // an expert is one item where there are enough for the warps
    const uint32_t parts = D == 0u || D >= warps ? 1u : tmin<uint32_t>((warps + D - 1u) / D, P.max_parts);
    const uint32_t ring = ptx::smem_u32(sm) + warp * warp_bytes, sslots = ring + RING * STAGE;
    const uint32_t dx = warps / parts, dp = warps - dx * parts;  // to a warp's next item: experts, parts

    // a position in the warp's list of steps: expert, first step, step, first pair of the
    // pass and of the expert, pairs of the expert, slot of its scales
    struct Pos {
        uint32_t x, j0, j, pb, first, cnt, slot;
    };
    auto enter = [&](Pos &p) {
        p.j = p.j0;
        p.pb = 0u;
        if (p.x < D) {
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
            p.x += dx;
            p.j0 += dp;
            if (p.j0 >= parts) {
                p.j0 -= parts;
                p.x++;
            }
            p.slot = p.slot + sslot == P.slots * sslot ? 0u : p.slot + sslot;
            enter(p);
        }
        return true;
    };
    // requests: the weights, at an item's start its scales, then h
    const uint8_t *w0 = nullptr;
    auto start_w = [&](const Pos &p) {
        if (p.x >= D) return;
        const size_t row = (size_t)experts[p.x] * P.H + row0;
        w0 = P.w2 + (row + r) * row_bytes;  // the lane's row of the first tile
        if (p.pb == 0u) {
            const uint8_t *s = P.s2 + row * srow, *b = P.a2 + row * srow;
            for (uint32_t o = lane * 16u; o < C * srow; o += 512u) {
                ptx::cp_async_16(sslots + p.slot + o, s + o, 16);
                if constexpr (affine(MODE)) ptx::cp_async_16(sslots + p.slot + C * srow + o, b + o, 16);
            }
        }
    };
    auto issue_w = [&](const Pos &p, uint32_t stage) {
        const uint32_t in = 4u * p.j + q < nu;
        const uint8_t *src = w0 + (in ? unit_byte<MODE>(4u * p.j + q) : 0u);
        const uint32_t st = ring + stage + lane * piece(MODE);
#pragma unroll
        for (uint32_t t = 0; t < 2 * T; t++, src += 8u * (size_t)row_bytes) copy_unit<MODE>(st + t * rows8(MODE), src, in);
    };
    uint32_t ho[PP];  // the pairs' offsets in hf
    auto start_h = [&](const Pos &p) {
        if (p.x >= D) return;
#pragma unroll
        for (uint32_t k = 0; k < PP; k++)
            ho[k] = p.pb + k < p.cnt ? (pairs[p.first + p.pb + k] & 0xFFFFu) * steps * HSTEP + lane * 16u : 0u;
    };
    auto issue_h = [&](const Pos &p, uint32_t stage) {
        const uint32_t st = ring + stage + HAT + lane * 16u;
        const uint8_t *src = P.hf + p.j * HSTEP;
#pragma unroll
        for (uint32_t k = 0; k < PP; k++)
#pragma unroll
            for (uint32_t o = 0; o < HSTEP; o += 512u)
                ptx::cp_async_16_if(p.pb + k < p.cnt && lane * 16u + o < HSTEP, st + k * HSTEP + o, src + ho[k] + o, 16);
    };

    Pos ahead{};
    {
        const uint32_t w = blockIdx.y * FEW_WARPS + warp;
        ahead.x = w / parts;
        ahead.j0 = w - ahead.x * parts;
    }
    enter(ahead);
    Pos at = ahead;
    // RING steps ahead of the arithmetic; P.slots covers the items that they reach
    start_w(ahead);
    uint32_t issued = 0;
    for (; issued < RING && ahead.x < D; issued++) {
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

    float acc[T][NB][2];
#pragma unroll
    for (int t = 0; t < T; t++)
#pragma unroll
        for (int n = 0; n < NB; n++) acc[t][n][0] = acc[t][n][1] = 0.f;
    Table<MODE> tab;
    tab.load(P.a2);
    const StepAt<NB> sa = step_at<NPL, NB>(ring + HAT, HSTEP, ptx::smem_u32(zeros), lane);
    uint32_t stage = 0;
    while (at.x < D) {
        wait_groups<RING - 1>();  // the oldest step: its weights came in an older group
        __syncwarp();             // and the other lanes' parts of the scales and of h
        const uint32_t u0 = tmin<uint32_t>(4u * at.j + 2u * (q & 1u), nu - 1u), u1 = tmin<uint32_t>(u0 + 1u, nu - 1u);
        const uint32_t i = scale_entry<MODE>(u0, P.gshift2);
        step<MODE, NPL, NB, T>(ring + stage + lane * piece(MODE), sslots + at.slot + r * srow, 16u * srow, 8u * srow,
                               C * srow, i, scale_entry<MODE>(u1, P.gshift2) - i, codes_before<MODE>(4u * at.j + q), tab,
                               sa, stage, lane, acc);
        const uint32_t pfirst = at.first + at.pb, pcnt = at.cnt - at.pb;
        const bool ended = advance(at);
        __syncwarp();  // every lane has read its stage and scales
        if (ahead.x < D) {
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
                float v[T][2];
#pragma unroll
                for (int t = 0; t < T; t++)
#pragma unroll
                    for (int h = 0; h < 2; h++) {
                        v[t][h] = acc[t][n][h] + __shfl_xor_sync(FULL, acc[t][n][h], 1);
                        if constexpr (NPL == 2) v[t][h] += __shfl_xor_sync(FULL, v[t][h], 2);
                        v[t][h] *= code_unit(MODE, NPL);
                        acc[t][n][h] = 0.f;
                    }
                // one pair at a time: two of them may be one token's
#pragma unroll
                for (uint32_t k = 0; k < 2u / NPL; k++) {
                    const uint32_t p = n * (2u / NPL) + k;
                    if (p < pcnt) {
                        if (q == 2u * k) {
                            float *y = ysm + (warp * P.m + (pairs[pfirst + p] >> 16)) * C + r;
#pragma unroll
                            for (int t = 0; t < T; t++) {
                                y[16 * t] += v[t][0];
                                y[16 * t + 8] += v[t][1];
                            }
                        }
                        __syncwarp();
                    }
                }
            }
        }
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
    __syncthreads();
    // the CTA's sums of (token, column) o
    auto own_sum = [&](uint32_t o) {
        float y = 0.f;
#pragma unroll
        for (uint32_t w = 0; w < FEW_WARPS; w++) y += ysm[w * P.m * C + o];
        return y;
    };
    if (P.split > 1u) {
        for (uint32_t o = tid; o < P.m * C; o += FEW_THREADS)
            P.partial[((size_t)blockIdx.y * P.m + o / C) * P.H + row0 + o % C] = own_sum(o);
        __threadfence();
        __syncthreads();
        if (tid == 0) last_s = atomicAdd(&P.arrived[blockIdx.x], 1u) + 1u == P.split;
        __syncthreads();
        if (!last_s) return;
        __threadfence();
    }
    for (uint32_t o = tid; o < P.m * C; o += FEW_THREADS) {
        const uint32_t t = o / C, c = row0 + o % C;
        const size_t oi = (size_t)t * P.H + c;
        float y = 0.f;
        if (P.split > 1u)
            for (uint32_t k = 0; k < P.split; k++) y += __ldcg(P.partial + (size_t)k * P.m * P.H + oi);
        else
            y = own_sum(o);
        if (P.bias2)
            for (uint32_t s = 0; s < P.S; s++) {
                const uint32_t e = ids_s[t * P.S + s];
                if (e != FULL)
                    y = fmaf(__ldg(P.weights + t * P.S + s), load_bias(P.bias2, P.bias2_dtype, (size_t)e * P.H + c), y);
            }
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

// Shared memory of the two kernels.
size_t up_bytes(int mode, uint32_t H, uint32_t groups, int planes, uint32_t blocks) {
    return FEW_WARPS * RING * UP_TILES * 2ull * rows8(mode) +
           (size_t)(2u * blocks / planes) * ((H / 32u + 3u) / 4u) * step_bytes(planes) +
           128ull * scale_bytes(mode, groups) * (affine(mode) ? 2u : 1u);
}
// mlp_down: an item has steps / max_parts steps or more; RING steps ahead reach so many more.
uint32_t down_parts(uint32_t steps) { return steps >= 4u ? steps / 2u : 1u; }
uint32_t down_slots(uint32_t steps) { return RING / (steps / down_parts(steps)) + 2u; }
size_t down_bytes(int mode, uint32_t I, uint32_t groups, int planes, uint32_t blocks, uint32_t tiles, uint32_t m) {
    const uint32_t slot = 16u * tiles * scale_bytes(mode, groups) * (affine(mode) ? 2u : 1u);
    return FEW_WARPS * (RING * (2ull * rows8(mode) * tiles + (2u * blocks / planes) * step_bytes(planes)) +
                        down_slots((I / 32u + 3u) / 4u) * (uint64_t)slot + 64ull * tiles * m);
}

template <int MODE, int PLANES, int NB>
cudaError_t up_t(const FewParams &P, cudaStream_t st) {
    const size_t smem = up_bytes(MODE, P.H, P.g1, PLANES, NB);
    auto kern = mlp_up<MODE, PLANES, NB>;
    static SmemSet smem_set;
    const cudaError_t e = ensure_dyn_smem(kern, smem, smem_set);
    if (e != cudaSuccess) return e;
    // about two waves of two CTAs an SM if every pair has an expert of its own: further
    // units of an expert follow in the same CTA, which saves it the prologue
    const uint32_t experts = tmin<uint32_t>(P.R, P.E);
    const uint32_t gx = tmin<uint32_t>((4u * SMS + experts - 1u) / experts, P.I / 32u);
    kern<<<dim3(gx, experts), FEW_THREADS, smem, st>>>(P);
    return cudaGetLastError();
}

template <int MODE, int NPL, int NB, int T>
cudaError_t down_t(FewParams P, cudaStream_t st) {
    const size_t smem = down_bytes(MODE, P.I, P.g2, NPL, NB, T, P.m);
    auto kern = mlp_down<MODE, NPL, NB, T>;
    static SmemSet smem_set;
    const cudaError_t e = ensure_dyn_smem(kern, smem, smem_set);
    if (e != cudaSuccess) return e;
    const uint32_t steps = (P.I / 32u + 3u) / 4u;
    P.max_parts = down_parts(steps);
    P.slots = down_slots(steps);
    // a programmatic dependent of mlp_up: it requests its weights while mlp_up runs and
    // waits (griddepcontrol.wait) before it reads h
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(P.H / (16u * T), P.split);
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

template <int MODE, int PLANES>
cudaError_t up_p(const FewParams &P, cudaStream_t st) {
    uint32_t blocks = blocks_a_pass(P, PLANES);
    while (blocks > 1u && up_bytes(MODE, P.H, P.g1, PLANES, blocks) > FEW_SMEM) blocks /= 2u;
    switch (blocks) {
        case 1: return up_t<MODE, PLANES, 1>(P, st);
        case 2: return up_t<MODE, PLANES, 2>(P, st);
        default: return up_t<MODE, PLANES, 4>(P, st);
    }
}

template <int MODE, int NPL>
cudaError_t down_p(const FewParams &P, cudaStream_t st) {
    // a token's columns on as many SMs as there are; else two tiles a warp, which
    // share a step's B registers and its loop
    if (P.R <= FEW_ALONE_R) return down_t<MODE, NPL, 1, 1>(P, st);
    uint32_t blocks = blocks_a_pass(P, NPL);
    while (blocks > 1u && down_bytes(MODE, P.I, P.g2, NPL, blocks, 2, P.m) > FEW_SMEM) blocks /= 2u;
    switch (blocks) {
        case 1: return down_t<MODE, NPL, 1, 2>(P, st);
        case 2: return down_t<MODE, NPL, 2, 2>(P, st);
        default: return down_t<MODE, NPL, 4, 2>(P, st);
    }
}

template <int MODE>
cudaError_t up_m(const FewParams &P, cudaStream_t st) {
    return x_planes(P.x_dtype) == 1 ? up_p<MODE, 1>(P, st) : up_p<MODE, 2>(P, st);
}
template <int MODE>
cudaError_t down_m(const FewParams &P, cudaStream_t st) {
    return h_planes(P.out_dtype) == 1 ? down_p<MODE, 1>(P, st) : down_p<MODE, 2>(P, st);
}

cudaError_t launch_up(const FewParams &P, int mode, cudaStream_t st) {
    switch (mode) {
        case M_A4: return up_m<M_A4>(P, st);
        case M_A4U: return up_m<M_A4U>(P, st);
        case M_A6: return up_m<M_A6>(P, st);
        case M_A8: return up_m<M_A8>(P, st);
        case M_NV: return up_m<M_NV>(P, st);
        case M_MX: return up_m<M_MX>(P, st);
        case M_CB2: return up_m<M_CB2>(P, st);
        case M_CB3: return up_m<M_CB3>(P, st);
        default: return up_m<M_CB4>(P, st);
    }
}

cudaError_t launch_down(const FewParams &P, int mode, cudaStream_t st) {
    switch (mode) {
        case M_A4: return down_m<M_A4>(P, st);
        case M_A4U: return down_m<M_A4U>(P, st);
        case M_A6: return down_m<M_A6>(P, st);
        case M_A8: return down_m<M_A8>(P, st);
        case M_NV: return down_m<M_NV>(P, st);
        case M_MX: return down_m<M_MX>(P, st);
        case M_CB2: return down_m<M_CB2>(P, st);
        case M_CB3: return down_m<M_CB3>(P, st);
        default: return down_m<M_CB4>(P, st);
    }
}

}  // namespace

// Bytes of h, of mlp_down's partial sums and of its counters.
static uint64_t few_h(uint64_t R, uint32_t inter) {
    return R * ((inter + 127ull) / 128ull) * step_bytes(h_planes(DT_F32));
}
static uint64_t few_partial(uint32_t m, uint32_t hidden) { return (uint64_t)MAX_SPLIT * m * hidden * 4ull; }

uint64_t mlp_few_workspace(uint32_t m, uint32_t hidden, uint32_t inter, uint32_t S) {
    // with more tokens than the kernels take, what fewer tokens in the same workspace need
    m = tmin<uint32_t>(m, FEW_MAX_TOKENS);
    const uint64_t R = tmin<uint64_t>((uint64_t)m * S, FEW_MAX_R);
    return few_h(R, inter) + few_partial(m, hidden) + (hidden / 16u + 1u) * 4ull;
}

// Whole 32-code units of 16 aligned bytes and scale groups of whole units in both
// projections, at most 512 pairs of at most 64 tokens, x in shared memory beside the
// ring.
bool mlp_few_supported(const MlpArgs &a) {
    const uint64_t R = (uint64_t)a.m * a.S;
    if (R > FEW_MAX_R || a.m > FEW_MAX_TOKENS || a.E > MOE_ROUTE_MAX_EXPERTS) return false;
    const int m1 = mode_of(*a.gate_up, a.hidden), m2 = mode_of(*a.down, a.inter);
    if (m1 < 0 || m2 < 0 || ((uintptr_t)a.x & 15u)) return false;
    return up_bytes(m1, a.hidden, a.hidden / a.gate_up->group_size, x_planes(a.x_dtype), 1) <= FEW_SMEM &&
           down_bytes(m2, a.inter, a.inter / a.down->group_size, h_planes(a.out_dtype), 1, 2, a.m) <=
               FEW_SMEM;
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
    const uint64_t at = few_h((uint64_t)a.m * a.S, a.inter);
    P.partial = (float *)(P.hf + at);
    P.arrived = (uint32_t *)(P.hf + at + few_partial(a.m, a.hidden));
    P.m = a.m; P.S = a.S; P.R = a.m * a.S; P.E = a.E; P.H = a.hidden; P.I = a.inter;
    P.g1 = a.hidden / a.gate_up->group_size; P.g2 = a.inter / a.down->group_size;
    P.gshift1 = log2_units(*a.gate_up); P.gshift2 = log2_units(*a.down);
    P.x_dtype = a.x_dtype; P.out_dtype = a.out_dtype; P.act = a.act;
    const int m1 = mode_of(*a.gate_up, a.hidden), m2 = mode_of(*a.down, a.inter);
    P.scale2_kind = m2 == M_NV;
    P.down_order = m2 == M_A4 || m2 == M_A4U ? 1 : m2 == M_A8 ? 2 : 0;
    P.rb1 = (uint32_t)moe_packed_row_bytes(a.gate_up->fmt, a.gate_up->bits, a.hidden);
    P.rb2 = (uint32_t)moe_packed_row_bytes(a.down->fmt, a.down->bits, a.inter);
    // mlp_down's CTAs: up to one wave of two an SM (a second wave would pay its prologue
    // again: 58 us against 62 with 3 and 4 CTAs a block of 88, 61 against 64 with 2 and 4
    // of 128); a token or two have too little work to be worth the join
    P.split = P.R <= FEW_ALONE_R ? 1u : tmin<uint32_t>(tmax<uint32_t>(2u * SMS / (P.H / 32u), 1u), MAX_SPLIT);
    const cudaError_t ce = launch_up(P, m1, st);
    return ce == cudaSuccess ? launch_down(P, m2, st) : ce;
}

}  // namespace moe
