// mlp_codes.cuh -- what the expert MLP's kernels on mma.sync share (mlp_few.cu,
// mlp_mid.cu): storage modes, packed codes to f16 pairs, and the images of x and h
// that stand against them.
#pragma once

#include "common.cuh"
#include "internal.h"
#include "ptx.cuh"

namespace moe {
namespace {

constexpr uint32_t FULL = 0xFFFFFFFFu;

// Storage as the kernels are specialised for it: affine 4 bits with groups of two units or
// more (one scale for the two units of a lane's accumulator columns) or of one unit,
// affine 6 and 8 bits, NVFP4 (two scales a unit), MXFP4, codebooks of 2, 3 and 4 bits.
enum Mode : int { M_A4, M_A4U, M_A6, M_A8, M_NV, M_MX, M_CB2, M_CB3, M_CB4 };
__host__ __device__ constexpr bool affine(int m) { return m == M_A4 || m == M_A4U || m == M_A6 || m == M_A8; }
__host__ __device__ constexpr bool codebook(int m) { return m == M_CB2 || m == M_CB3 || m == M_CB4; }

// A lane's unit of 32 codes of one row, as it is copied: pieces of 4, 8 or 16 bytes.
__host__ __device__ constexpr uint32_t piece(int m) { return m == M_CB3 ? 4u : m == M_A6 || m == M_CB2 ? 8u : 16u; }
__host__ __device__ constexpr uint32_t pieces(int m) { return m == M_CB3 ? 4u : m == M_A6 ? 3u : m == M_A8 ? 2u : 1u; }
constexpr int words(int m) { return (int)(piece(m) * pieces(m) / 4u); }
// The units of 8 rows in the ring: [piece][lane].
__host__ __device__ constexpr uint32_t rows8(int m) { return 32u * piece(m) * pieces(m); }

// One step of one pair's x or h, 128 values: planes [plane][unit 4][64 bytes], then
// (factor, sum of the values) of each unit, f32.
__host__ __device__ constexpr uint32_t step_bytes(int planes) { return (uint32_t)planes * 256u + 32u; }

__device__ __forceinline__ uint4 lds128(uint32_t a) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a));
    return v;
}
__device__ __forceinline__ uint2 lds64(uint32_t a) {
    uint2 v;
    asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a));
    return v;
}
__device__ __forceinline__ uint32_t lds32(uint32_t a) {
    uint32_t v;
    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(a));
    return v;
}
__device__ __forceinline__ uint32_t lds16(uint32_t a) {
    uint16_t v;
    asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(a));
    return v;
}
__device__ __forceinline__ uint32_t lds8(uint32_t a) {
    uint32_t v;
    asm volatile("ld.shared.u8 %0, [%1];" : "=r"(v) : "r"(a));
    return v;
}

// --------------------------------------------------------------------- codes

// Byte of a row at which unit u's pieces begin (3-bit words hold 10 codes: its first word).
template <int MODE>
__device__ __forceinline__ uint32_t unit_byte(uint32_t u) {
    if constexpr (MODE == M_CB3) return (32u * u / 10u) * 4u;
    else return u * piece(MODE) * pieces(MODE);
}

// Copies one unit (zeros where `in` is 0: nothing is read then).
template <int MODE>
__device__ __forceinline__ void copy_unit(uint32_t dst, const uint8_t *src, uint32_t in) {
#pragma unroll
    for (uint32_t k = 0; k < pieces(MODE); k++) {
        const uint32_t d = dst + k * 32u * piece(MODE);
        const uint8_t *s = src + k * piece(MODE);
        if constexpr (piece(MODE) == 16u) ptx::cp_async_16(d, s, in ? 16u : 0u);
        else if constexpr (piece(MODE) == 8u) ptx::cp_async_8(d, s, in ? 8u : 0u);
        else ptx::cp_async_4(d, s, in ? 4u : 0u);
    }
}

template <int MODE>
__device__ __forceinline__ void load_unit(uint32_t a, uint32_t (&w)[words(MODE)]) {
#pragma unroll
    for (uint32_t k = 0; k < pieces(MODE); k++) {
        const uint32_t at = a + k * 32u * piece(MODE);
        if constexpr (piece(MODE) == 16u) {
            const uint4 v = lds128(at);
            w[4 * k] = v.x; w[4 * k + 1] = v.y; w[4 * k + 2] = v.z; w[4 * k + 3] = v.w;
        } else if constexpr (piece(MODE) == 8u) {
            const uint2 v = lds64(at);
            w[2 * k] = v.x; w[2 * k + 1] = v.y;
        } else {
            w[k] = lds32(at);
        }
    }
}

// Byte permutation as the instruction does it: bit 3 of a selector repeats the byte's sign
// (__byte_perm drops it, with an instruction of its own).
__device__ __forceinline__ uint32_t prmt(uint32_t a, uint32_t b, uint32_t sel) {
    uint32_t d;
    asm("prmt.b32 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(sel));
    return d;
}

// The f16 codebook's low and high bytes, as the byte permutation looks them up.
template <int MODE>
struct Table {
    static constexpr int N = MODE == M_CB4 ? 4 : MODE == M_CB3 ? 2 : 1;
    uint32_t lo[N], hi[N];
    __device__ __forceinline__ void load(const uint8_t *cb) {
        if constexpr (codebook(MODE)) {
#pragma unroll
            for (int i = 0; i < N; i++) {
                lo[i] = hi[i] = 0u;
#pragma unroll
                for (int k = 0; k < 4; k++) {
                    const uint32_t v = __ldg((const unsigned short *)cb + 4 * i + k);
                    lo[i] |= (v & 0xFFu) << (8 * k);
                    hi[i] |= (v >> 8) << (8 * k);
                }
            }
        }
    }
    // Four codes, one in each nibble of the low half of `sel`, as two f16 pairs.
    __device__ __forceinline__ void look(uint32_t sel, uint32_t &p, uint32_t &q) const {
        uint32_t l, h;
        if constexpr (N < 4) {
            l = prmt(lo[0], lo[N - 1], sel);
            h = prmt(hi[0], hi[N - 1], sel);
        } else {
            const uint32_t s7 = sel & 0x7777u, s8 = sel & 0x8888u;
            const uint32_t upper = prmt(0x00008000u, 0u, s8 | (s8 >> 3));  // 0xFF where the code is 8 or more
            l = (prmt(lo[0], lo[1], s7) & ~upper) | (prmt(lo[2], lo[3], s7) & upper);
            h = (prmt(hi[0], hi[1], s7) & ~upper) | (prmt(hi[2], hi[3], s7) & upper);
        }
        p = prmt(l, h, 0x5140);
        q = prmt(l, h, 0x7362);
    }
};

// A unit's words before they are expanded: 3-bit words of 10 codes joined into 96 bits
// from the unit's first code on (word_codes = codes before it in its first word).
template <int MODE>
__device__ __forceinline__ void join_words(uint32_t (&w)[words(MODE)], uint32_t word_codes) {
    if constexpr (MODE == M_CB3) {
        const uint32_t m = 0x3FFFFFFFu, a = w[0] & m, b = w[1] & m, c = w[2] & m, d = w[3] & m;
        const uint32_t x0 = a | (b << 30), x1 = (b >> 2) | (c << 28), x2 = (c >> 4) | (d << 26), x3 = d >> 6;
        const uint32_t s = 3u * word_codes;
        w[0] = __funnelshift_r(x0, x1, s);
        w[1] = __funnelshift_r(x1, x2, s);
        w[2] = __funnelshift_r(x2, x3, s);
    }
}

// Codes 8 t .. 8 t + 7 of a unit as f16 pairs:
//   affine, as integers times 2^-24: 4 bits (0, 4), (1, 5), (2, 6), (3, 7), the second and
//   fourth pair 16 times that; 8 bits (0, 2), (1, 3), (4, 6), (5, 7); 6 bits in order
//   E2M1 and codebook values in order: (0, 1), (2, 3), (4, 5), (6, 7)
// CENTRED (affine, for f32 results): the integers less the middle of their range, which the
// bias makes up for. The tensor core cuts products off 24 bits below the largest term,
// and sums of codes that are all positive lose several times more of what is left once
// the bias is added (2.3e-6 of an f32 result against 64 bits).
template <int MODE, bool CENTRED>
__device__ __forceinline__ void expand(const uint32_t (&w)[words(MODE)], int t, const Table<MODE> &T, uint32_t (&p)[4]) {
    if constexpr (MODE == M_A4 || MODE == M_A4U) {
        p[0] = w[t] & 0x000F000Fu;
        p[1] = w[t] & 0x00F000F0u;
        p[2] = (w[t] >> 8) & 0x000F000Fu;
        p[3] = (w[t] >> 8) & 0x00F000F0u;
    } else if constexpr (MODE == M_A8) {
#pragma unroll
        for (int i = 0; i < 2; i++) {
            p[2 * i] = w[2 * t + i] & 0x00FF00FFu;
            p[2 * i + 1] = (w[2 * t + i] >> 8) & 0x00FF00FFu;
        }
    } else if constexpr (MODE == M_A6) {
#pragma unroll
        for (int i = 0; i < 4; i++) {
            const int bit = 48 * t + 12 * i, k = bit / 32, s = bit % 32;
            const uint32_t v = s <= 20 ? w[k] >> s : __funnelshift_r(w[k], w[k + 1 < 6 ? k + 1 : k], s);
            p[i] = (v & 0x3Fu) | ((v << 10) & 0x003F0000u);
        }
    } else if constexpr (MODE == M_NV || MODE == M_MX) {
        asm("{.reg .b8 a, b, c, d; mov.b32 {a, b, c, d}, %4; cvt.rn.f16x2.e2m1x2 %0, a; cvt.rn.f16x2.e2m1x2 %1, b; "
            "cvt.rn.f16x2.e2m1x2 %2, c; cvt.rn.f16x2.e2m1x2 %3, d;}"
            : "=r"(p[0]), "=r"(p[1]), "=r"(p[2]), "=r"(p[3])
            : "r"(w[t]));
    } else {
        // the codes spread to nibbles: halves, quarters and eighths apart, other bits last
        uint32_t n;
        if constexpr (MODE == M_CB4) {
            n = w[t];
        } else if constexpr (MODE == M_CB2) {
            const uint32_t v = t & 1 ? w[t / 2] >> 16 : w[t / 2];
            n = (v & 0xFFu) | ((v << 8) & ~0xFFu);
            n = (n & 0x00FF00FFu) | ((n << 4) & 0xFF00FF00u);
            n = ((n & 0x0F0F0F0Fu) | ((n << 2) & 0xF0F0F0F0u)) & 0x33333333u;
        } else {
            const uint32_t v = t == 0 ? w[0] : t == 1 ? __funnelshift_r(w[0], w[1], 24)
                             : t == 2 ? __funnelshift_r(w[1], w[2], 16) : w[2] >> 8;
            n = (v & 0xFFFu) | ((v << 4) & ~0xFFFu);
            n = (n & 0x00FF00FFu) | ((n << 2) & 0xFF00FF00u);
            n = ((n & 0x0F0F0F0Fu) | ((n << 1) & 0xF0F0F0F0u)) & 0x77777777u;
        }
        T.look(n, p[0], p[1]);
        T.look(n >> 16, p[2], p[3]);
    }
    if constexpr (CENTRED) {
        // 0x6400 | c is 1024 + c (1024 + 16 c a nibble higher); exact
        constexpr uint32_t less = MODE == M_A8 ? 0xE480E480u : MODE == M_A6 ? 0xE420E420u : 0xE408E408u;
#pragma unroll
        for (int i = 0; i < 4; i++) {
            const uint32_t v = p[i] | 0x64006400u;
            if ((MODE == M_A4 || MODE == M_A4U) && i % 2 == 1)
                asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(p[i]) : "r"(v), "r"(0x2C002C00u), "r"(0xD480D480u));
            else
                asm("add.rn.f16x2 %0, %1, %2;" : "=r"(p[i]) : "r"(v), "r"(less));
        }
    }
}
constexpr bool centred(int mode, int planes) { return affine(mode) && planes == 2; }
constexpr float middle(int mode) { return mode == M_A8 ? 128.f : mode == M_A6 ? 32.f : 8.f; }
// What expand()'s values have to be multiplied by: the sums of x that meet the biases are
// divided by it and the results multiplied, since a unit's factor times 2^24 can leave f32.
constexpr float code_unit(int mode, int planes) { return affine(mode) && !centred(mode, planes) ? 16777216.f : 1.f; }

// Order of x against expand()'s pairs: 0 as it stands, 1 as 4-bit affine words part it
// (where not centred with a sixteenth of the values that meet the 16-fold pairs), 2 as
// 8-bit words do.
constexpr int order_of(int mode) { return mode == M_A4 || mode == M_A4U ? 1 : mode == M_A8 ? 2 : 0; }
// Place of value c of a unit among its 32 f16 values.
__device__ __forceinline__ uint32_t b_place(int order, uint32_t c) {
    return order == 1 ? (c & ~7u) + 2u * (c & 3u) + ((c >> 2) & 1u)
         : order == 2 ? (c & ~3u) + 2u * (c & 1u) + ((c >> 1) & 1u) : c;
}

__device__ __forceinline__ void mma(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                    uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// The first of a sum.
__device__ __forceinline__ void mma0(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                     uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
        : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
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
__host__ __device__ constexpr uint32_t scale_bytes(int mode, uint32_t groups) {
    return affine(mode) || codebook(mode) ? groups * 2u : groups;
}

// Byte of unit u's entry in a row's scales.
template <int MODE>
__device__ __forceinline__ uint32_t scale_entry(uint32_t u, uint32_t gshift) {
    return affine(MODE) || codebook(MODE) ? (u >> gshift) * 2u : MODE == M_NV ? 2u * u : u;
}

template <int N>
__device__ __forceinline__ void wait_groups() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// Four consecutive x values.
__device__ __forceinline__ float4 load_x4(const void *x, int dt, size_t i) {
    if (dt == DT_F32) return __ldg((const float4 *)((const float *)x + i));
    const uint2 v = __ldg((const uint2 *)((const uint16_t *)x + i));
    if (dt == DT_BF16)
        return make_float4(__uint_as_float(v.x << 16), __uint_as_float(v.x & 0xFFFF0000u), __uint_as_float(v.y << 16),
                           __uint_as_float(v.y & 0xFFFF0000u));
    return make_float4(f16_bits_to_f32(v.x & 0xFFFFu), f16_bits_to_f32(v.x >> 16), f16_bits_to_f32(v.y & 0xFFFFu),
                       f16_bits_to_f32(v.y >> 16));
}

// Four values of lane l (4l .. 4l+3 of a step) times `scale`, in the order of MODE's codes.
template <int MODE, int PLANES>
__device__ __forceinline__ float4 in_order(float4 v, float scale, uint32_t lane) {
    if constexpr (order_of(MODE) == 1) {
        // a word's pairs are (0, 4), (1, 5) for the even lane and (2, 6), (3, 7) for the odd one
        const bool odd = lane & 1u;
        const float s0 = odd ? v.x : v.z, s1 = odd ? v.y : v.w;
        const float r0 = __shfl_xor_sync(FULL, s0, 1), r1 = __shfl_xor_sync(FULL, s1, 1);
        const float sixteenth = centred(MODE, PLANES) ? scale : scale * 0.0625f;
        return odd ? make_float4(r0 * scale, v.z * scale, r1 * sixteenth, v.w * sixteenth)
                   : make_float4(v.x * scale, r0 * scale, v.y * sixteenth, r1 * sixteenth);
    } else if constexpr (order_of(MODE) == 2) {
        return make_float4(v.x * scale, v.z * scale, v.y * scale, v.w * scale);
    } else {
        return make_float4(v.x * scale, v.y * scale, v.z * scale, v.w * scale);
    }
}

// A warp writes one step image: lane l holds values 4l .. 4l+3 (unit l / 8).
template <int MODE, int PLANES>
__device__ __forceinline__ void write_step(uint8_t *dst, float4 v, uint32_t lane) {
    const uint32_t M = 0x7FFFFFFFu;
    uint32_t mb = max(max(__float_as_uint(v.x) & M, __float_as_uint(v.y) & M),
                      max(__float_as_uint(v.z) & M, __float_as_uint(v.w) & M));
    float sum = (v.x + v.y) + (v.z + v.w);
#pragma unroll
    for (int d = 1; d < 8; d <<= 1) {
        mb = max(mb, __shfl_xor_sync(FULL, mb, d));
        if constexpr (affine(MODE)) sum += __shfl_xor_sync(FULL, sum, d);
    }
    float scale, factor;
    unit_scale(mb, scale, factor);
    v = in_order<MODE, PLANES>(v, scale, lane);
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

// The mode of a projection, or -1.
inline int mode_of(const moe_expert_weights &w, uint32_t k) {
    const int kind = kind_of((int)w.fmt, (int)w.bits);
    if (k % 32u != 0 || (((uintptr_t)w.packed | (uintptr_t)w.scales) & 15u)) return -1;
    if (kind == K_NVFP4) return ((uintptr_t)w.aux & 3u) ? -1 : M_NV;
    if (kind == K_MXFP4) return M_MX;
    const uint32_t u = w.group_size / 32u;  // units a group
    if (w.group_size % 32u != 0 || (u & (u - 1u)) != 0) return -1;
    if (w.fmt == MOE_FMT_AFFINE) {
        if ((uintptr_t)w.aux & 15u) return -1;
        return kind == K_AFF4 ? (u == 1u ? M_A4U : M_A4) : kind == K_AFF6 ? M_A6 : M_A8;
    }
    if ((uintptr_t)w.aux & 1u) return -1;
    return kind == K_CB2 ? M_CB2 : kind == K_CB3 ? M_CB3 : M_CB4;
}

// log2(units of 32 codes a scale group).
inline uint32_t log2_units(const moe_expert_weights &w) {
    uint32_t s = 0;
    while ((32u << s) < w.group_size) s++;
    return s;
}

}  // namespace
}  // namespace moe
