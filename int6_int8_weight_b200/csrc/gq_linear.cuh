// gq_linear.cuh -- the layer product over tiled int6 / int8 weights with bias,
// activation and residual in its epilogue, and the same grouped by expert
// (definitions in include/gq.h).
#pragma once

#include "gq_gemm.cuh"

namespace gq {

// ------------------------------------------------------------ tile layout --
//
// A weight [N, K] is padded to tiles of 128 rows and blocks of 64 columns
// (code 0).  Block (rt, kb) is 6144 (int6) or 8192 (int8) contiguous bytes,
// [chunk][row][16 bytes], blocks kb-major within a row tile: a K range of a tile
// is one bulk copy, and a warp whose lane r reads row r's chunk reads 512
// consecutive bytes of shared memory.
//   int6: a row's 64 codes are four groups of 16; a group is three words of
//   eight pairs p_j = u(2j) | u(2j + 1) << 16, u = q + 32:
//     word i = p_i | p_(3+i) << 6 | (nibbles at bits 12..15 and 28..31), i = 0..2;
//     the nibbles of words 0 and 1 are the low four bits of pairs 6 and 7,
//     that of word 2 their high two bits (pair 6 in its low half).
//   So pairs 0..2 leave a word with one mask, 3..5 with a shift and a mask.
//   int8: bytes of codes 0, 2, 1, 3 of each four (two's complement): a word
//   is a pair at bits 0..7 / 16..23 and one at bits 8..15 / 24..31.
constexpr int kLinRows = 128;
constexpr int kLinK = 64;

__host__ __device__ constexpr int lin_block_bytes(int qbits) { return kLinRows * (qbits == 6 ? 48 : 64); }

// One thread per row of a block: 64 codes of the packed row in, 48 / 64 bytes of
// the tile out.  The packed rows may start at any byte, so they are read byte by
// byte, and the lanes of a warp read a row pitch apart: bound by those loads
// (16384 x 16384: 1420 us int6, 966 int8; its bytes once in and out would be 61
// and 82).  It runs once per weight, when that is exported or loaded.
__global__ void __launch_bounds__(kLinRows) tile_weight_kernel(const uint8_t* __restrict__ packed, int64_t N, int64_t K,
                                                               int64_t prb, int qbits, int64_t kbs, uint8_t* tiles) {
    const int64_t block = blockIdx.x;                      // (expert, row tile, column block)
    const int64_t rts = (N + kLinRows - 1) / kLinRows;
    const int64_t kb = block % kbs, rt = block / kbs % rts, e = block / kbs / rts;
    const int64_t n = rt * kLinRows + threadIdx.x;
    const uint8_t* row = packed + (e * N + n) * prb;
    auto code = [&](int i) -> uint32_t {                   // two's complement, the field's bits only
        const int64_t k = kb * kLinK + i;
        if (n >= N || k >= K) return 0u;
        if (qbits == 8) return row[k];
        const int64_t bit = 6 * k, at = bit >> 3;
        const uint32_t lo = row[at], hi = (bit & 7) > 2 ? row[at + 1] : 0u;
        return ((lo | hi << 8) >> (bit & 7)) & 63u;
    };
    uint4* out = reinterpret_cast<uint4*>(tiles + block * lin_block_bytes(qbits)) + threadIdx.x;
    uint32_t w[16];
    if (qbits == 8) {
#pragma unroll
        for (int j = 0; j < 16; ++j)
            w[j] = code(4 * j) | code(4 * j + 2) << 8 | code(4 * j + 1) << 16 | code(4 * j + 3) << 24;
    } else {
#pragma unroll
        for (int g = 0; g < 4; ++g) {
            uint32_t p[8];
#pragma unroll
            for (int j = 0; j < 8; ++j)
                p[j] = (code(16 * g + 2 * j) ^ 32u) | (code(16 * g + 2 * j + 1) ^ 32u) << 16;
            w[3 * g] = p[0] | p[3] << 6 | (p[6] & 0x000F000Fu) << 12;
            w[3 * g + 1] = p[1] | p[4] << 6 | (p[7] & 0x000F000Fu) << 12;
            w[3 * g + 2] = p[2] | p[5] << 6 | (p[6] >> 4 & 0x00030003u) << 12 | (p[7] >> 4 & 0x00030003u) << 14;
        }
        w[12] = w[13] = w[14] = w[15] = 0u;
    }
    const int chunks = qbits == 6 ? 3 : 4;
    for (int c = 0; c < chunks; ++c)
        out[c * kLinRows] = make_uint4(w[4 * c], w[4 * c + 1], w[4 * c + 2], w[4 * c + 3]);
}

// ----------------------------------------------------------------- codes --

// a * b + c on bf16 pairs (one instruction; the pair subtraction is several).
__device__ __forceinline__ uint32_t lin_fma2(uint32_t a, uint32_t b, uint32_t c) {
    uint32_t r;
    asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(b), "r"(c));
    return r;
}

// (a & b) | c in one instruction: written out, because with two constants the
// compiler takes a masking and an or-ing one.
__device__ __forceinline__ uint32_t lin_and_or(uint32_t a, uint32_t b, uint32_t c) {
    uint32_t r;
    asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(r) : "r"(a), "r"(b), "r"(c));
    return r;
}

// The 8 pairs of codes of one int6 group (three words) as bf16x2 integers.  A
// 6-bit field u in a half's low bits under 0x4300 is the bf16 number 128 + u; less
// 160 it is q, exactly.
__device__ __forceinline__ void lin_codes6(uint32_t w0, uint32_t w1, uint32_t w2, uint32_t* o) {
    constexpr uint32_t m = 0x003F003Fu, h = 0x43004300u, one = 0x3F803F80u, s = 0xC320C320u;
    o[0] = lin_fma2(lin_and_or(w0, m, h), one, s);
    o[1] = lin_fma2(lin_and_or(w1, m, h), one, s);
    o[2] = lin_fma2(lin_and_or(w2, m, h), one, s);
    o[3] = lin_fma2(lin_and_or(w0 >> 6, m, h), one, s);
    o[4] = lin_fma2(lin_and_or(w1 >> 6, m, h), one, s);
    o[5] = lin_fma2(lin_and_or(w2 >> 6, m, h), one, s);
    o[6] = lin_fma2(lin_and_or(w0 >> 12, 0x000F000Fu, lin_and_or(w2 >> 8, 0x00300030u, h)), one, s);
    o[7] = lin_fma2(lin_and_or(w1 >> 12, 0x000F000Fu, lin_and_or(w2 >> 10, 0x00300030u, h)), one, s);
}

// The two pairs of an int8 word: the low seven bits give 128 + low, the sign bit
// under 0x4300 is 128 or 256, and their difference is q, exactly.
__device__ __forceinline__ void lin_codes8(uint32_t w, uint32_t& a, uint32_t& b) {
    constexpr uint32_t m = 0x007F007Fu, t = 0x00800080u, h = 0x43004300u, minus = 0xBF80BF80u;
    const uint32_t v = w >> 8;
    a = lin_fma2(lin_and_or(w, t, h), minus, lin_and_or(w, m, h));
    b = lin_fma2(lin_and_or(v, t, h), minus, lin_and_or(v, m, h));
}

// -------------------------------------------------------------- epilogue --

struct LinEpi {
    const void* bias;            // [N] (grouped: [E, N]) or null
    const void* residual;        // [M, ldr] or null
    void* y;                     // [M, ldy]
    int64_t ldr, ldy;
    int32_t bias_bf16, residual_bf16, y_bf16, act;
};

// Two values in a register pair: sums and products of both in one issue.
struct LinF2 {
    uint64_t r;
    __device__ __forceinline__ LinF2(float a, float b) { asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b)); }
    __device__ __forceinline__ explicit LinF2(float a) : LinF2(a, a) {}
    __device__ __forceinline__ void out(float& a, float& b) const {
        asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(r));
    }
};
__device__ __forceinline__ LinF2 lin_fma(LinF2 a, LinF2 b, LinF2 c) {
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(a.r) : "l"(a.r), "l"(b.r), "l"(c.r));
    return a;
}
__device__ __forceinline__ LinF2 operator*(LinF2 a, LinF2 b) {
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(a.r) : "l"(a.r), "l"(b.r));
    return a;
}
__device__ __forceinline__ LinF2 operator+(LinF2 a, LinF2 b) {
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(a.r) : "l"(a.r), "l"(b.r));
    return a;
}

// From the special function unit: 2^a and 1 / a.
__device__ __forceinline__ float lin_exp2(float a) {
    asm("ex2.approx.ftz.f32 %0, %0;" : "+f"(a));
    return a;
}
__device__ __forceinline__ float lin_rcp(float a) {
    asm("rcp.approx.ftz.f32 %0, %0;" : "+f"(a));
    return a;
}
__device__ __forceinline__ float lin_relu(float a) {       // NaN stays NaN
    asm("max.NaN.f32 %0, %0, 0f00000000;" : "+f"(a));
    return a;
}

// 1 / (1 + 2^a): 0 and 1 where 2^a over- or underflows.
__device__ __forceinline__ LinF2 lin_sigmoid2(LinF2 a) {
    float x, y;
    a.out(x, y);
    (LinF2(lin_exp2(x), lin_exp2(y)) + LinF2(1.0f)).out(x, y);
    return LinF2(lin_rcp(x), lin_rcp(y));
}

// The normal distribution function: 1 - Phi(|x|) = t (b1 + t (b2 + .. + t b5)) e^(-x^2 / 2), t = 1 / (1 + q |x|), the
// approximation of Hastings (Abramowitz and Stegun 7.1.26, with half its coefficients), absolute error below 1e-7.
__device__ __forceinline__ LinF2 lin_phi(float x, float y) {
    const LinF2 z(x, y), t(lin_rcp(__fmaf_rn(0.23164189f, fabsf(x), 1.0f)), lin_rcp(__fmaf_rn(0.23164189f, fabsf(y), 1.0f)));
    float ex, ey, px, py, ux, uy;
    (z * z * LinF2(-0.72134752f)).out(ex, ey);
    LinF2 p = lin_fma(t, LinF2(0.5307027145f), LinF2(-0.7265760135f));
    p = lin_fma(t, p, LinF2(0.7107068705f));
    p = lin_fma(t, p, LinF2(-0.142248368f));
    p = lin_fma(t, p, LinF2(0.127414796f));
    p = p * t * LinF2(lin_exp2(ex), lin_exp2(ey));
    p.out(px, py);
    lin_fma(p, LinF2(-1.0f), LinF2(1.0f)).out(ux, uy);
    return LinF2(x < 0.0f ? px : ux, y < 0.0f ? py : uy);
}

// N (even) values through the activation, in place, two at a time.  NaN stays NaN.
// silu and the gelus take the exponential and the quotient from the special
// function unit and the normal distribution from a polynomial, for binary32 Y
// too: chosen for the pair kernel, whose epilogue shares the issue slots with the
// conversion (M 4096, N = K = 8192 with gelu_tanh: 9 % less time than with expf and a
// division, forms of its own for a residual and for none included).  Measured over
// [-30, 30] against binary64, in 2^-24 max(|z|, 1): at most 2.8, 2.9 and 2.8 for silu, gelu and
// gelu_tanh (torch's binary32 forms: 2.0 each).  In the negative tail silu is off by
// 5e-7 of its value at -6 and by 2e-6 at -30, gelu_tanh by 3e-6 at -6, and gelu,
// whose error is absolute, by 4e-3 at -6.
template <int N>
__device__ __forceinline__ void lin_act(float (&z)[N], int act) {
    // one test of `act` for all of them, and a loop of its own for each
    auto each = [&](auto f) {
#pragma unroll
        for (int i = 0; i < N; i += 2) f(z[i], z[i + 1]).out(z[i], z[i + 1]);
    };
    switch (act) {
        case GQ_ACT_RELU: each([](float x, float y) { return LinF2(lin_relu(x), lin_relu(y)); }); break;
        case GQ_ACT_RELU2:
            each([](float x, float y) {
                const LinF2 r(lin_relu(x), lin_relu(y));
                return r * r;
            });
            break;
        case GQ_ACT_LEAKY_RELU2:
            each([](float x, float y) {
                float hx, hy;
                (LinF2(x, y) * LinF2(0.5f)).out(hx, hy);
                const LinF2 r(x < 0.0f ? hx : x, y < 0.0f ? hy : y);
                return r * r;
            });
            break;
        case GQ_ACT_SILU:
            each([](float x, float y) { return LinF2(x, y) * lin_sigmoid2(LinF2(x, y) * LinF2(-1.4426950408889634f)); });
            break;
        case GQ_ACT_GELU: each([](float x, float y) { return LinF2(x, y) * lin_phi(x, y); }); break;
        case GQ_ACT_GELU_TANH:
            // tanh(w) + 1 = 2 sigmoid(2 w), 2 w = 2 sqrt(2 / pi) (x + 0.044715 x^3), here times -log2(e)
            each([](float x, float y) {
                const LinF2 z(x, y);
                return z * lin_sigmoid2(z * lin_fma(z * z, LinF2(-0.10294324f), LinF2(-2.3022082f)));
            });
            break;
        default: break;
    }
}

__device__ __forceinline__ float lin_elem(const void* p, int64_t i, int bf16) {
    return bf16 ? bf16_bits_to_float(static_cast<const uint16_t*>(p)[i]) : static_cast<const float*>(p)[i];
}

// N rows of Y from row m on, column n (the first `count` of them), from their
// sums, the column's scale and bias.  The residual (RES: there is one) is read
// before anything is written (it may be Y itself), all N loads in flight while the
// activation is worked out.  Whole runs are told apart from the last rows of a
// tile: a test and a branch for each element cost as much as the rest.
template <bool RES, bool WHOLE, int N>
__device__ __forceinline__ void lin_rows_out(const LinEpi& E, float (&v)[N], int count, float s, float b, int64_t m,
                                             int64_t n) {
    uint32_t r[N];
    if constexpr (RES) {
        if (E.residual_bf16) {
            const uint16_t* p = static_cast<const uint16_t*>(E.residual) + m * E.ldr + n;
#pragma unroll
            for (int i = 0; i < N; ++i, p += E.ldr) r[i] = WHOLE || i < count ? (uint32_t)*p : 0u;
        } else {
            const uint32_t* p = static_cast<const uint32_t*>(E.residual) + m * E.ldr + n;
#pragma unroll
            for (int i = 0; i < N; ++i, p += E.ldr) r[i] = WHOLE || i < count ? *p : 0u;
        }
    }
#pragma unroll
    for (int i = 0; i < N; i += 2)                         // (b is 0 without a bias)
        lin_fma(LinF2(v[i], v[i + 1]), LinF2(s), LinF2(b)).out(v[i], v[i + 1]);
    lin_act(v, E.act);
    if constexpr (RES) {
        const int shift = E.residual_bf16 ? 16 : 0;
#pragma unroll
        for (int i = 0; i < N; i += 2)
            (LinF2(v[i], v[i + 1]) + LinF2(__uint_as_float(r[i] << shift), __uint_as_float(r[i + 1] << shift)))
                .out(v[i], v[i + 1]);
    }
    if (E.y_bf16) {
        uint16_t* p = static_cast<uint16_t*>(E.y) + m * E.ldy + n;
#pragma unroll
        for (int i = 0; i < N; ++i, p += E.ldy)
            if (WHOLE || i < count) *p = float_to_bf16_bits(v[i]);
    } else {
        float* p = static_cast<float*>(E.y) + m * E.ldy + n;
#pragma unroll
        for (int i = 0; i < N; ++i, p += E.ldy)
            if (WHOLE || i < count) *p = v[i];
    }
}

template <bool RES, int N>
__device__ __forceinline__ void lin_finish_as(const LinEpi& E, float (&v)[N], int count, float s, float b, int64_t m,
                                           int64_t n) {
    if (count >= N) lin_rows_out<RES, true>(E, v, count, s, b, m, n);
    else lin_rows_out<RES, false>(E, v, count, s, b, m, n);
}

template <int N>
__device__ __forceinline__ void lin_finish(const LinEpi& E, float (&v)[N], int count, float s, float b, int64_t m,
                                           int64_t n) {
    if (E.residual) lin_finish_as<true>(E, v, count, s, b, m, n);
    else lin_finish_as<false>(E, v, count, s, b, m, n);
}

struct LinParams {
    CUtensorMap tmap_x;          // X [M, K] bf16, box {64, tokens of a tile}, SWIZZLE_128B
    const uint8_t* tiles;
    const uint16_t* scale;
    const int32_t* offsets;      // [E + 1] or null (one weight)
    int32_t* status;
    int64_t M, N, E;
    int32_t kbs, rts;            // column blocks, row tiles of a weight
    int32_t log_split;           // 2^this blocks (a cluster) share a tile's column blocks
    int32_t stages;              // ring depth
    uint32_t idesc;
    LinEpi epi;
};

// ------------------------------------------------------------- PTX glue --

// Bulk copy of `bytes` (a multiple of 16) global -> this block's shared memory.
__device__ __forceinline__ void lin_bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
                 "l"(src), "r"(bytes), "r"(bar)
                 : "memory");
}

__device__ __forceinline__ void lin_tmem_ld8(uint32_t taddr, float (&f)[8]) {
    uint32_t v[8];
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7])
                 : "r"(taddr));
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = __uint_as_float(v[i]);
}

// Columns taddr + 64 j .. + 15 (j = 0 .. 3) of this thread's lane into 64
// registers; one asm block, so that nothing touches them before they are there.
__device__ __forceinline__ void lin_tmem_drain(uint32_t taddr, float (&v)[16][4]) {
#define GQ_LD16 "tcgen05.ld.sync.aligned.32x32b.x16.b32 {"
#define GQ_OUT4(j) "=f"(v[j][0]), "=f"(v[j][1]), "=f"(v[j][2]), "=f"(v[j][3])
    asm volatile(GQ_LD16 "%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%64];\n\t"
                 GQ_LD16 "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%65];\n\t"
                 GQ_LD16 "%32, %33, %34, %35, %36, %37, %38, %39, %40, %41, %42, %43, %44, %45, %46, %47}, [%66];\n\t"
                 GQ_LD16 "%48, %49, %50, %51, %52, %53, %54, %55, %56, %57, %58, %59, %60, %61, %62, %63}, [%67];\n\t"
                 "tcgen05.wait::ld.sync.aligned;"
                 : GQ_OUT4(0), GQ_OUT4(1), GQ_OUT4(2), GQ_OUT4(3), GQ_OUT4(4), GQ_OUT4(5), GQ_OUT4(6), GQ_OUT4(7),
                   GQ_OUT4(8), GQ_OUT4(9), GQ_OUT4(10), GQ_OUT4(11), GQ_OUT4(12), GQ_OUT4(13), GQ_OUT4(14), GQ_OUT4(15)
                 : "r"(taddr), "r"(taddr + 64u), "r"(taddr + 128u), "r"(taddr + 192u)
                 : "memory");
#undef GQ_LD16
#undef GQ_OUT4
}

// v[a ..] = v[b ..], 16 values, as moves that stay where they are written: from
// assignments the compiler makes copies of the whole array on every way through
// the pair kernel's loop (8192 rows over 32 experts: 5 % more time, 20 moves for
// each element of Y).
__device__ __forceinline__ void lin_move16(float (&v)[16][4], int a, int b) {
#define GQ_OUT4(j) "=f"(v[a + j][0]), "=f"(v[a + j][1]), "=f"(v[a + j][2]), "=f"(v[a + j][3])
#define GQ_IN4(j) "f"(v[b + j][0]), "f"(v[b + j][1]), "f"(v[b + j][2]), "f"(v[b + j][3])
    asm volatile("mov.b32 %0, %16;\n\tmov.b32 %1, %17;\n\tmov.b32 %2, %18;\n\tmov.b32 %3, %19;\n\t"
                 "mov.b32 %4, %20;\n\tmov.b32 %5, %21;\n\tmov.b32 %6, %22;\n\tmov.b32 %7, %23;\n\t"
                 "mov.b32 %8, %24;\n\tmov.b32 %9, %25;\n\tmov.b32 %10, %26;\n\tmov.b32 %11, %27;\n\t"
                 "mov.b32 %12, %28;\n\tmov.b32 %13, %29;\n\tmov.b32 %14, %30;\n\tmov.b32 %15, %31;"
                 : GQ_OUT4(0), GQ_OUT4(1), GQ_OUT4(2), GQ_OUT4(3)
                 : GQ_IN4(0), GQ_IN4(1), GQ_IN4(2), GQ_IN4(3));
#undef GQ_OUT4
#undef GQ_IN4
}

// The binary32 at shared address `addr` of block `rank` of the cluster.
__device__ __forceinline__ float lin_ld_peer(uint32_t addr, uint32_t rank) {
    float f;
    asm volatile("{\n\t.reg .b32 a;\n\tmapa.shared::cluster.u32 a, %1, %2;\n\tld.shared::cluster.f32 %0, [a];\n\t}"
                 : "=f"(f)
                 : "r"(addr), "r"(rank)
                 : "memory");
    return f;
}

// The 4 MMAs (K = 16 each) of one column block, over CTAS blocks: as
// g_mma_stage_ts, but from the low word of X's shared memory descriptor, and all
// its arguments the same in every lane, so that the compiler can keep them in
// uniform registers.  The issuing warp is the narrow place of a stage's way: with
// descriptors put together anew for each column block M 16, N = K = 16384 takes 6 % more time.
__device__ __forceinline__ uint32_t lin_desc_low(uint32_t addr) { return (uint32_t)g_smem_desc(addr); }
template <int CTAS>
__device__ __forceinline__ void lin_mma(uint32_t d_tmem, uint32_t a_tmem, uint32_t b_low, uint32_t idesc,
                                        uint32_t accumulate) {
#define GQ_MMA(kind)                                                                                                   \
    asm volatile(                                                                                                      \
        "{\n\t.reg .pred p, e;\n\t.reg .b64 b0, b1, b2, b3;\n\t"                                                      \
        "mov.b64 b0, {%5, %10};\n\tmov.b64 b1, {%6, %10};\n\tmov.b64 b2, {%7, %10};\n\tmov.b64 b3, {%8, %10};\n\t"     \
        "setp.ne.b32 p, %9, 0;\n\t"                                                                                    \
        "elect.sync _|e, 0xffffffff;\n\t"                                                                              \
        "@e tcgen05.mma." kind ".kind::f16 [%0], [%1], b0, %11, p;\n\t"                                                \
        "@e tcgen05.mma." kind ".kind::f16 [%0], [%2], b1, %11, 1;\n\t"                                                \
        "@e tcgen05.mma." kind ".kind::f16 [%0], [%3], b2, %11, 1;\n\t"                                                \
        "@e tcgen05.mma." kind ".kind::f16 [%0], [%4], b3, %11, 1;\n\t"                                                \
        "}\n" ::"r"(d_tmem),                                                                                           \
        "r"(a_tmem), "r"(a_tmem + 8u), "r"(a_tmem + 16u), "r"(a_tmem + 24u), "r"(b_low), "r"(b_low + 2u),              \
        "r"(b_low + 4u), "r"(b_low + 6u), "r"(accumulate), "r"((uint32_t)(g_smem_desc(0u) >> 32)), "r"(idesc)          \
        : "memory")
    if constexpr (CTAS == 2) GQ_MMA("cta_group::2");
    else GQ_MMA("cta_group::1");
#undef GQ_MMA
}
// A value that every lane holds, for the compiler to know it.
__device__ __forceinline__ uint32_t lin_uniform(uint32_t x) { return __reduce_or_sync(0xffffffffu, x); }

// Four consecutive rows of a column from the S blocks' sums at shared address
// `at`, added in rank order: all 4 S loads are on their way before the first
// addition.
template <int S>
__device__ __forceinline__ void lin_gather(float (&v)[4], uint32_t at) {
    float t[S][4];
#pragma unroll
    for (int q = 0; q < S; ++q)
#pragma unroll
        for (int i = 0; i < 4; ++i) t[q][i] = lin_ld_peer(at + 512u * i, (uint32_t)q);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[i] = t[0][i];
#pragma unroll
        for (int q = 1; q < S; ++q) v[i] += t[q][i];
    }
}

__device__ __forceinline__ void lin_cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// g_wait with its first test kept apart from the loop: what follows a wait that
// is over at once is a branch (the ALU is what the conversion is bound by).
__device__ __forceinline__ bool lin_wait(uint32_t bar, uint32_t parity) {
    if (__builtin_expect(g_try_wait(bar, parity), 1)) return true;
    return g_wait(bar, parity);
}

// One weight row's 64 codes of a block (its 16-byte chunks lie 2048 bytes apart
// at shared address `src`) into the 32 TMEM columns at `taddr` of this
// thread's lane: column j holds k = 2j and 2j + 1 as bf16.
template <int QB>
__device__ __forceinline__ void lin_codes_to_tmem(uint32_t src, uint32_t taddr) {
    auto chunk = [&](int c, uint32_t* w) {
        asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3])
                     : "r"(src + 16u * kLinRows * c)
                     : "memory");
    };
    uint32_t w[16], o[16];
    chunk(0, w);
    chunk(1, w + 4);
    if constexpr (QB == 6) {
        chunk(2, w + 8);
        lin_codes6(w[0], w[1], w[2], o);
        lin_codes6(w[3], w[4], w[5], o + 8);
        g_tmem_st16(taddr, o);
        lin_codes6(w[6], w[7], w[8], o);
        lin_codes6(w[9], w[10], w[11], o + 8);
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) lin_codes8(w[j], o[2 * j], o[2 * j + 1]);
        chunk(2, w);
        chunk(3, w + 4);
        g_tmem_st16(taddr, o);
#pragma unroll
        for (int j = 0; j < 8; ++j) lin_codes8(w[j], o[2 * j], o[2 * j + 1]);
    }
    g_tmem_st16(taddr + 16u, o);
}

// ------------------------------------------------------------- scheduling --

// linear_kernel is launched with programmatic stream serialization: a block
// lets the next kernel's blocks take the SMs as they come free (every block of
// this one is running by then), and before its first access to memory that
// another kernel may have written, or may still read, it waits until all kernels
// before it are done and their writes visible.  What precedes is only a block's
// own preparation (barriers, tensor memory).
__device__ __forceinline__ void lin_release_next() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void lin_wait_previous() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// A unit of work: one tile of 128 weight rows by up to NT consecutive rows of X
// of one expert.
struct LinUnit {
    int32_t e, m0, m1;           // expert, rows [m0, m1) of X
    int32_t rt;                  // row tile
    int32_t bad;                 // an offset out of order or range was met
};

// Tile j of the rows [a, b): as few tiles as NT allows, of even size (a multiple
// of 32, the granularity of the pair kernel's MMAs).
template <int NT>
__device__ __forceinline__ void lin_cut(LinUnit& u, int a, int b, int j) {
    const unsigned rows = (unsigned)(b - a), n = (rows + NT - 1u) / NT;
    const int step = NT < 32 ? NT : (int)((rows + n - 1u) / n + 31u & ~31u);
    u.m0 = a + j * step;
    u.m1 = min(b - u.m0, step) + u.m0;
}

// Token tiles of the whole batch (one warp): none where an offset is out of order or range, since ranges that overlap
// could add up to any number of tiles.
template <int NT>
__device__ __forceinline__ int lin_total(const LinParams& P) {
    if (!P.offsets) return (int)((P.M + NT - 1) / NT);
    unsigned sum = 0;
    bool ok = true;
    for (int e = threadIdx.x & 31; e < (int)P.E; e += 32) {
        const int p = __ldg(P.offsets + e), q = __ldg(P.offsets + e + 1);
        if (p >= 0 && q >= p && q <= (int)P.M)
            sum += ((unsigned)(q - p) + NT - 1u) / NT;
        else
            ok = false;
    }
    sum = __reduce_add_sync(0xffffffffu, sum);
    if (__all_sync(0xffffffffu, ok)) return (int)sum;
    if (threadIdx.x == 0 && P.status) atomicOr(reinterpret_cast<unsigned int*>(P.status), 0x8u);
    return 0;
}

// The MMAs' N for a unit of the pair kernel: its rows in steps of 32.
__device__ __forceinline__ int lin_cols(const LinUnit& u) { return u.m1 - u.m0 + 31 & ~31; }

// The inclusive prefix sum of the lanes' tile counts, held at 2^30 (only offsets that are out of order could carry it
// past the rows' number).
__device__ __forceinline__ int lin_prefix(int n) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int o = __shfl_up_sync(0xffffffffu, n, d);
        if (lane >= d) n = (int)min((unsigned)n + (unsigned)o, 1u << 30);
    }
    return n;
}

// Unit `tt` of the token tiles (expert-major) found by one warp: every lane counts
// the tiles of its share of the experts, all its loads in flight, then the lanes look
// at one expert each of the share that holds the unit (8 rows, N 512, K 2048, 512
// experts: 6.7 us, and 10.6 with 32 experts after the other).  m0 = m1 past the last.
template <int NT>
__device__ __forceinline__ LinUnit lin_find(const LinParams& P, int tt) {
    LinUnit u{0, 0, 0, 0, 0};
    const int M = (int)P.M, E = (int)P.E;
    if (!P.offsets) {
        lin_cut<NT>(u, 0, M, tt);
        return u;
    }
    const int lane = threadIdx.x & 31;
    int first = 0, last = E, before = 0;                   // experts to look at, tiles of those before them
    if (E > 32) {
        const int share = (E + 31) >> 5, a = min(lane * share, E), b = min(a + share, E);
        int sum = 0, p = __ldg(P.offsets + a);
        bool ok = true;
#pragma unroll 8
        for (int e = a; e < b; ++e) {
            const int q = __ldg(P.offsets + e + 1);
            const bool in = p >= 0 && q >= p && q <= M;
            ok = ok && in;
            sum = (int)min((unsigned)sum + (in ? ((unsigned)(q - p) + NT - 1u) / NT : 0u), 1u << 30);
            p = q;
        }
        if (!__all_sync(0xffffffffu, ok)) u.bad = 1;
        const int at = lin_prefix(sum);
        const uint32_t who = __ballot_sync(0xffffffffu, sum > 0 && tt < at && tt >= at - sum);
        if (!who) return u;
        const int l = __ffs(who) - 1;
        before = __shfl_sync(0xffffffffu, at - sum, l);
        first = l * share;
        last = min(first + share, E);
    }
    for (int e0 = first; e0 < last; e0 += 32) {
        const int e = e0 + lane;
        int a = 0, b = 0;
        bool ok = true;
        if (e < last) {
            const int p = __ldg(P.offsets + e), q = __ldg(P.offsets + e + 1);
            ok = p >= 0 && q >= p && q <= M;
            a = ok ? p : 0;
            b = ok ? q : 0;
        }
        if (!__all_sync(0xffffffffu, ok)) u.bad = 1;
        const int n = (int)(((unsigned)(b - a) + NT - 1u) / NT);
        const int at = (int)min((unsigned)before + (unsigned)lin_prefix(n), 1u << 30);   // tiles up to and with this expert's
        const uint32_t who = __ballot_sync(0xffffffffu, n > 0 && tt < at && tt >= at - n);
        if (who) {
            const int l = __ffs(who) - 1;
            u.e = e0 + l;
            lin_cut<NT>(u, __shfl_sync(0xffffffffu, a, l), __shfl_sync(0xffffffffu, b, l),
                        __shfl_sync(0xffffffffu, tt - (at - n), l));
            return u;
        }
        before = __shfl_sync(0xffffffffu, at, 31);
    }
    return u;
}

// ----------------------------------------------------------------- kernel --
//
// One block per unit, or a cluster of 2^log_split blocks that share its column
// blocks.  The weight tile is the MMA's A operand, M = 128, and the tokens its B
// operand, N = NT: a decode step pays for no padding of the tokens to 128 rows.
// Warps:
//   0       copies: a stage is two column blocks (128 of K): their codes by one
//           bulk copy, the X tiles by TMA
//   1       TMEM allocation, then the MMAs
//   2 ..    codes -> bf16 integers in TMEM (A operand): groups of four warps
//           that take the stages (or their halves) in turn, thread r of a group
//           weight row r; then the epilogue
// Shared memory carries codes and X only, and a code costs about 1.6
// instructions on the way (masks, shifts, one exact subtraction per pair); the
// row scale waits until the epilogue.
// With a split the blocks put their sums into their own shared memory, and
// after a cluster barrier each finishes its share of the elements, adding the
// blocks' sums in rank order.
constexpr int kLinMaxStages = 8;

template <int QB, int NT>
struct LinShape {
    static constexpr uint32_t x_block = NT * 128u;                       // one column block of X
    static constexpr uint32_t c_block = lin_block_bytes(QB);
    static constexpr uint32_t stage = 2 * (x_block + c_block);
    static constexpr uint32_t acc_cols = NT <= 64 ? 64 : NT;
    static constexpr uint32_t slots = (256 - acc_cols) / 64;             // stages of A in TMEM
    // Conversion groups of four warps, and how many of them share a stage.  Two whole-stage groups wait and hand over
    // half as often as four half-stage ones (M 16, N = K = 16384: 8 % less time); with 128 tokens the MMAs
    // leave only two slots, and four groups hide more (M 4096, N = K = 8192 in this kernel: 19 % less).
    static constexpr int groups = NT <= 64 ? 2 : 4, parts = NT <= 64 ? 1 : 2;
    static constexpr int threads = 64 + 128 * groups;
    static constexpr uint32_t bars = 8 * (2 * kLinMaxStages + 2 * 4 + 2) + 64;
    static constexpr int smem(int stages) { return 1024 + stages * (int)stage + (int)bars; }
};

template <int QB, int NT>
__global__ void __launch_bounds__(LinShape<QB, NT>::threads, 2) linear_kernel(const __grid_constant__ LinParams P) {
    using S = LinShape<QB, NT>;
    extern __shared__ unsigned char g_smem[];
    __shared__ LinUnit s_unit;
    const uint32_t base = (g_smem_u32(g_smem) + 1023u) & ~1023u;
    const int D = P.stages;
    const uint32_t bars = base + (uint32_t)D * S::stage;
    auto full = [&](int s) { return bars + 8u * s; };
    auto empty = [&](int s) { return bars + 8u * (kLinMaxStages + s); };
    auto wready = [&](int t) { return bars + 8u * (2 * kLinMaxStages + t); };
    auto tfree = [&](int t) { return bars + 8u * (2 * kLinMaxStages + 4 + t); };
    const uint32_t acc_full = bars + 8u * (2 * kLinMaxStages + 8);
    const uint32_t tmem_slot = acc_full + 8u;
    auto x_tile = [&](int s, int j) { return base + (uint32_t)s * S::stage + j * S::x_block; };
    auto c_tile = [&](int s, int j) { return base + (uint32_t)s * S::stage + 2 * S::x_block + j * S::c_block; };

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    // the split is a power of two; 32-bit arithmetic throughout (a 64-bit division costs more than a block of codes)
    const uint32_t split = 1u << P.log_split, rank = blockIdx.x & (split - 1u);
    const uint32_t index = blockIdx.x >> P.log_split;      // unit: token tile by row tile, row tiles fastest
    if (warp == 2) {
        lin_wait_previous();
        const uint32_t tt = index / (uint32_t)P.rts;
        LinUnit u = lin_find<NT>(P, (int)tt);
        u.rt = (int32_t)(index - tt * (uint32_t)P.rts);
        if (lane == 0) {
            s_unit = u;
            if (u.bad && P.status) atomicOr(reinterpret_cast<unsigned int*>(P.status), 0x8u);
        }
    } else if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 256;" ::"r"(tmem_slot) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    } else if (threadIdx.x == 0) {
        for (int s = 0; s < D; ++s) {
            g_bar_init(full(s), 1);
            g_bar_init(empty(s), 1);
        }
        for (int t = 0; t < (int)S::slots; ++t) {
            g_bar_init(wready(t), 4 * S::parts);
            g_bar_init(tfree(t), 1);
        }
        g_bar_init(acc_full, 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&P.tmap_x)) : "memory");
    }
    asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
    __syncthreads();
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
    uint32_t tmem;
    asm volatile("ld.shared.b32 %0, [%1];" : "=r"(tmem) : "r"(tmem_slot) : "memory");
    lin_wait_previous();
    lin_release_next();
    const LinUnit u = s_unit;
    const int mv = u.m1 - u.m0;                            // rows of X in the unit
    // this block's column blocks, two a stage
    const int kb0 = (int)((uint32_t)P.kbs * rank >> P.log_split), kb1 = (int)((uint32_t)P.kbs * (rank + 1) >> P.log_split);
    const int stages = mv > 0 ? (kb1 - kb0 + 1) / 2 : 0;
    // the weight row that this thread's elements of Y belong to, in either form of the epilogue
    const int64_t n = (int64_t)u.rt * kLinRows + (split > 1 ? threadIdx.x & 127 : 32 * (warp & 3) + lane);
    float sc = 0.0f, bi = 0.0f;
    if (mv > 0 && n < P.N) {
        sc = __half2float(__ushort_as_half(P.scale[(int64_t)u.e * P.N + n]));
        if (P.epi.bias) bi = lin_elem(P.epi.bias, (int64_t)u.e * P.N + n, P.epi.bias_bf16);
    }
    bool ok = true;
    if (warp == 0) {
        const uint8_t* codes = P.tiles + (((int64_t)u.e * P.rts + u.rt) * P.kbs + kb0) * (int64_t)S::c_block;
        int s = 0;
        uint32_t ph = 0u;
        int issued = 0;
        for (; issued < stages; ++issued) {
            if (issued >= D && !g_wait_warp(empty(s), ph ^ 1u)) {
                ok = false;
                break;
            }
            if (lane == 0) {
                const int kb = kb0 + 2 * issued, n = min(2, kb1 - kb);
                g_arrive_tx(full(s), (uint32_t)n * (S::x_block + S::c_block));
                lin_bulk_load(c_tile(s, 0), codes, (uint32_t)n * S::c_block, full(s));
                codes += n * S::c_block;
                for (int j = 0; j < n; ++j)
                    g_tma_load_2d(x_tile(s, j), &P.tmap_x, (kb + j) * kLinK, (int)u.m0, full(s));
            }
            if (++s == D) {
                s = 0;
                ph ^= 1u;
            }
        }
        // no copy may still be landing when the block reuses or leaves its memory
        for (int q = max(0, issued - D); q < issued; ++q)
            if (!g_wait_warp(full(q % D), (uint32_t)((q / D) & 1))) ok = false;
    } else if (warp == 1) {
        int s = 0, t = 0;
        uint32_t tph = 0u;
        const uint32_t acc = lin_uniform(tmem), b_low = lin_desc_low(base);
        for (int i = 0; i < stages; ++i) {
            // the warps that announce the codes have waited for the stage's copies, X among them
            if (!g_wait_warp(wready(t), tph)) {
                ok = false;
                break;
            }
            asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
            const uint32_t a = acc + S::acc_cols + 64u * t, b = b_low + (uint32_t)s * (S::stage >> 4);
            lin_mma<1>(acc, a, b, P.idesc, i ? 1u : 0u);
            if (2 * i + 1 < kb1 - kb0) lin_mma<1>(acc, a + 32u, b + (S::x_block >> 4), P.idesc, 1u);
            g_commit(empty(s));
            g_commit(tfree(t));
            if (++s == D) s = 0;
            if (++t == (int)S::slots) {
                t = 0;
                tph ^= 1u;
            }
        }
        g_commit(acc_full);                                // every MMA issued is done
        if (!g_wait_warp(acc_full, 0u)) ok = false;
    } else {
        const int grp = (warp - 2) >> 2, quarter = warp & 3, r = 32 * quarter + lane;
        const uint32_t lanes = (uint32_t)(32 * quarter) << 16;
        constexpr int kStep = S::groups / S::parts;       // stages from one of a group's to its next
        static_assert(kStep <= (int)S::slots, "the parity tests below");
        const int part = grp % S::parts;
        int s = grp / S::parts, t = s;
        uint32_t ph = 0u, tph = 0u;
        for (int i = s; i < stages; i += kStep) {
            // The slot first: once stage i - slots is done, stage i - stages (no later, the ring being at least as deep)
            // has landed, so a parity test of full(s) cannot take an older phase for this one; nor can one of
            // tfree(t), since the group's last stage was at most `slots` before.
            if ((i >= (int)S::slots && !lin_wait(tfree(t), tph ^ 1u)) || !lin_wait(full(s), ph)) ok = false;
            if (!__all_sync(0xffffffffu, ok)) {
                ok = false;
                break;
            }
            asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
            const uint32_t src = c_tile(s, part) + 16u * r, dst = tmem + lanes + S::acc_cols + 64u * t + 32u * part;
            const int n = kb1 - kb0 - 2 * i - part;        // blocks from this one on
            if (n > 0) lin_codes_to_tmem<QB>(src, dst);
            if (S::parts == 1 && n > 1) lin_codes_to_tmem<QB>(src + S::c_block, dst + 32u);
            asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
            asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
            __syncwarp();
            if (lane == 0) g_arrive(wready(t));
            if ((s += kStep) >= D) {
                s -= D;
                ph ^= 1u;
            }
            if ((t += kStep) >= (int)S::slots) {
                t -= (int)S::slots;
                tph ^= 1u;
            }
        }
        if (!g_wait_warp(acc_full, 0u)) ok = false;
        asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
        if (stages > 0) {
            for (int c0 = 8 * grp; c0 < mv; c0 += 8 * S::groups) {   // the groups take turns of 8 tokens
                float v[8];
                lin_tmem_ld8(tmem + lanes + (uint32_t)c0, v);
                if (split > 1) {
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        if (c0 + i < mv)
                            asm volatile("st.shared.f32 [%0], %1;" ::"r"(
                                             base + 4u * (uint32_t)((c0 + i) * kLinRows + r)),
                                         "f"(v[i])
                                         : "memory");
                } else if (n < P.N) {
                    lin_finish(P.epi, v, mv - c0, sc, bi, (int64_t)u.m0 + c0, n);
                }
                __syncwarp();                              // the next load wants the warp whole again
            }
        }
    }
    if (!ok && lane == 0 && P.status) atomicOr(reinterpret_cast<unsigned int*>(P.status), 0x4u);
    __syncwarp();
    if (split > 1 && mv > 0) {                           // the same in every block of the cluster
        lin_cluster_sync();
        // four rows of Y by 128 threads at a time over the cluster; a thread keeps its column
        constexpr int kLines = S::threads / kLinRows;
        const int line = (int)threadIdx.x / kLinRows;
        if (line < kLines && n < P.N)
            for (int c = 4 * ((int)rank * kLines + line); c < mv; c += 4 * (int)split * kLines) {
                const uint32_t at = base + 4u * (uint32_t)(c * kLinRows + ((int)threadIdx.x & 127));
                float v[4];                                // (rows past mv: whatever the sums' memory holds, not stored)
                if (split == 2) lin_gather<2>(v, at);
                else if (split == 4) lin_gather<4>(v, at);
                else lin_gather<8>(v, at);
                lin_finish(P.epi, v, mv - c, sc, bi, (int64_t)u.m0 + c, n);
            }
        __syncwarp();                                      // lanes past the last column skipped the loop
        lin_cluster_sync();                                // its memory is read until here
    }
    asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
    __syncthreads();
    if (warp == 1) {
        asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 256;" ::"r"(tmem) : "memory");
    }
}

// ------------------------------------------------------------ pair kernel --
//
// Many rows: two blocks of a cluster (on two SMs) work on one tile of 256
// weight rows by up to 256 rows of X with cta_group::2 MMAs (M = 256).  Each
// converts its own 128 weight rows into its own tensor memory and loads half of
// the X tile; the MMAs, issued by block 0, read both halves.  So a code is
// converted once per 256 tokens and X crosses to each SM half as often as with
// one block per tile: per SM and column block 16 KB of X and 6 KB of codes
// against 512 cycles of MMAs.
// Persistent: a pair takes every pairs-th unit.  TMEM: 256 columns of sums, 256
// for four stages of A.  Warp 0 copies, warp 1 of block 0 issues the MMAs (2 and
// 3 only make up the warpgroup that hands its registers over), 4 .. 19 convert,
// four groups of four, group g the stages that are g modulo 4.  The groups convert
// three stages ahead into the next unit (1500 cycles of MMAs), take the finished
// sums into registers as soon as the last MMA is done (64 a thread; that frees
// them for the next unit's MMAs), and apply the epilogue in four runs of 16
// tokens, each between two stages of conversion, so that the MMAs never wait for
// a whole epilogue.  Block 0's barriers gather both blocks' conversions (wready)
// and drains (acc_empty); the MMAs' commits arrive on both blocks' barriers.
// Bound: the tensor pipe.  M 4096, N = K = 8192, bias, gelu_tanh and residual: 368 us
// (1495 TFLOP/s) on a cool device, 435 in a loop that the power cap holds at 1.33 GHz.
constexpr int kPairNT = 256;
constexpr int kPairThreads = 128 + 512;
constexpr int kPairRoleRegs = 32, kPairConvRegs = 112;     // 4 * 32 + 16 * 112 = 20 * 96: what the block is launched with
constexpr int kPairSlots = 4;
constexpr int kPairMaxStages = 5;

template <int QB>
struct PairShape {
    static constexpr uint32_t x_block = kPairNT / 2 * 128u;              // half a tile's column block of X
    static constexpr uint32_t c_block = lin_block_bytes(QB);
    static constexpr uint32_t stage = 2 * (x_block + c_block);
    static constexpr uint32_t bars = 8 * (2 * kPairMaxStages + 2 * kPairSlots + 2) + 64;
    static constexpr int smem(int stages) { return 1024 + stages * (int)stage + (int)bars; }
    static constexpr int stages = smem(kPairMaxStages) <= 232448 ? kPairMaxStages : 4;
    static_assert(smem(stages) <= 232448 && stages >= kPairSlots, "the conversion's parity tests need stages >= slots");
};

// Arrive on block 0's barrier at the same place as `bar`.  What it announces is
// in tensor memory (ordered by the tcgen05 fences) or came by a copy that the
// arriving thread has waited for, so the default scope will do; a release at
// cluster scope waits for the thread's earlier stores to reach the other SM
// (M 4096, N = K = 8192: 7 % more time).
__device__ __forceinline__ void lin_arrive_lead(uint32_t bar) {
    asm volatile("{\n\t.reg .b32 a;\n\tmapa.shared::cluster.u32 a, %0, 0;\n\t"
                 "mbarrier.arrive.shared::cluster.b64 _, [a];\n\t}" ::"r"(bar)
                 : "memory");
}

// Arrive on `bar` of both blocks once the MMAs issued so far are done.
__device__ __forceinline__ void lin_commit_both(uint32_t bar) {
    asm volatile(
        "{\n\t.reg .pred e;\n\telect.sync _|e, 0xffffffff;\n\t"
        "@e tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;\n\t}\n" ::"r"(
            bar),
        "h"((uint16_t)3)
        : "memory");
}

template <int QB>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kPairThreads, 1)
    linear_pair_kernel(const __grid_constant__ LinParams P) {
    using S = PairShape<QB>;
    constexpr int D = S::stages;
    extern __shared__ unsigned char g_smem[];
    const uint32_t base = (g_smem_u32(g_smem) + 1023u) & ~1023u;
    const uint32_t bars = base + D * S::stage;
    auto full = [&](int s) { return bars + 8u * s; };
    auto empty = [&](int s) { return bars + 8u * (kPairMaxStages + s); };
    auto wready = [&](int t) { return bars + 8u * (2 * kPairMaxStages + t); };
    auto tfree = [&](int t) { return bars + 8u * (2 * kPairMaxStages + kPairSlots + t); };
    const uint32_t acc_full = bars + 8u * (2 * kPairMaxStages + 2 * kPairSlots), acc_empty = acc_full + 8u;
    const uint32_t tmem_slot = acc_full + 16u;
    auto x_tile = [&](int s, int j) { return base + (uint32_t)s * S::stage + j * S::x_block; };
    auto c_tile = [&](int s, int j) { return base + (uint32_t)s * S::stage + 2 * S::x_block + j * S::c_block; };

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = blockIdx.x & 1u;                 // cluster dimension (2, 1, 1)
    const int pair = (int)(blockIdx.x >> 1), pairs = (int)(gridDim.x >> 1);
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(tmem_slot) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    } else if (threadIdx.x == 0) {
        for (int s = 0; s < D; ++s) {
            g_bar_init(full(s), 1);
            g_bar_init(empty(s), 1);
        }
        for (int t = 0; t < kPairSlots; ++t) {
            g_bar_init(wready(t), 8);                      // the four warps of a group in each block
            g_bar_init(tfree(t), 1);
        }
        g_bar_init(acc_full, 1);
        g_bar_init(acc_empty, 32);                         // the sixteen conversion warps of each block
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&P.tmap_x)) : "memory");
    }
    const int tts = lin_total<kPairNT>(P);                 // token tiles
    asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
    __syncthreads();
    lin_cluster_sync();                                    // the other block's barriers are ready
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
    uint32_t tmem;
    asm volatile("ld.shared.b32 %0, [%1];" : "=r"(tmem) : "r"(tmem_slot) : "memory");

    const int rtps = (P.rts + 1) >> 1, units = tts * rtps;
    const int stages = (P.kbs + 1) >> 1;
    bool ok = true;
    int seq = 0;                                           // stages so far, over all units
    if (warp < 4) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kPairRoleRegs));
    if (warp == 0) {
        int s = 0;
        uint32_t ph = 0u;
        for (int q = pair; q < units && ok; q += pairs) {
            const LinUnit u = lin_find<kPairNT>(P, q / rtps);
            // the weight rows past the last tile are converted from the last tile's codes and never stored
            const int rt = min(2 * (q % rtps) + (int)rank, P.rts - 1);
            const uint8_t* codes = P.tiles + ((int64_t)u.e * P.rts + rt) * P.kbs * S::c_block;
            const int m0 = u.m0 + (int)rank * (lin_cols(u) >> 1);
            if (P.epi.residual) {                          // the unit's share of the residual into L2
                const int es = P.epi.residual_bf16 ? 2 : 4;
                const int64_t n0 = (int64_t)(2 * (q % rtps) + (int)rank) * kLinRows, n1 = min(n0 + kLinRows, P.N);
                for (int m = u.m0 + lane; m < u.m1; m += 32)
                    for (int64_t n = n0; n < n1; n += 128 / es)
                        asm volatile("prefetch.global.L2 [%0];" ::"l"(static_cast<const char*>(P.epi.residual) +
                                                                      (m * P.epi.ldr + n) * es));
                __syncwarp();
            }
            for (int i = 0; i < stages; ++i, ++seq) {
                if (seq >= D && !g_wait_warp(empty(s), ph ^ 1u)) {
                    ok = false;
                    break;
                }
                if (lane == 0) {
                    const int kb = 2 * i, n = min(2, P.kbs - kb);
                    g_arrive_tx(full(s), (uint32_t)n * (S::x_block + S::c_block));
                    lin_bulk_load(c_tile(s, 0), codes + (int64_t)kb * S::c_block, (uint32_t)n * S::c_block, full(s));
                    for (int j = 0; j < n; ++j)
                        g_tma_load_2d(x_tile(s, j), &P.tmap_x, (kb + j) * kLinK, m0, full(s));
                }
                if (++s == D) {
                    s = 0;
                    ph ^= 1u;
                }
            }
        }
        // every copy has landed and every commit has arrived before the block may leave
        for (int q = max(0, seq - D); q < seq; ++q)
            if (!g_wait_warp(full(q % D), (uint32_t)((q / D) & 1)) || !g_wait_warp(empty(q % D), (uint32_t)((q / D) & 1)))
                ok = false;
    } else if (warp == 1) {
        int s = 0, t = 0, done = 0;
        uint32_t tph = 0u;
        const uint32_t acc = lin_uniform(tmem), b_low = lin_desc_low(base);
        for (int q = pair; q < units && ok; q += pairs, ++done) {
            const LinUnit u = lin_find<kPairNT>(P, q / rtps);
            if (rank == 0) {
                const uint32_t idesc = gemm_idesc(2 * kLinRows, (uint32_t)lin_cols(u));
                if (done > 0 && !g_wait_warp(acc_empty, (uint32_t)(done - 1) & 1u)) ok = false;
                for (int i = 0; i < stages && ok; ++i) {
                    if (!g_wait_warp(wready(t), tph)) {    // (and with it for both blocks' copies, as in linear_kernel)
                        ok = false;
                        break;
                    }
                    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
                    const uint32_t a = acc + kPairNT + 64u * t, b = b_low + (uint32_t)s * (S::stage >> 4);
                    lin_mma<2>(acc, a, b, idesc, i ? 1u : 0u);
                    if (2 * i + 1 < P.kbs) lin_mma<2>(acc, a + 32u, b + (S::x_block >> 4), idesc, 1u);
                    lin_commit_both(empty(s));
                    lin_commit_both(tfree(t));
                    if (++s == D) s = 0;
                    if (++t == kPairSlots) {
                        t = 0;
                        tph ^= 1u;
                    }
                }
                lin_commit_both(acc_full);
            }
            seq += stages;
        }
        for (int q = max(0, seq - kPairSlots); q < seq; ++q)
            if (!g_wait_warp(tfree(q % kPairSlots), (uint32_t)((q / kPairSlots) & 1))) ok = false;
    } else if (warp >= 4) {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kPairConvRegs));
        const int grp = (warp - 4) >> 2, quarter = warp & 3, r = 32 * quarter + lane;
        const uint32_t lanes = (uint32_t)(32 * quarter) << 16;
        // Group grp takes the stages with seq % 4 == grp, so its TMEM slot is always the same.  (Everything that can be
        // worked out again is: the drained sums take 64 of a thread's 112 registers.)
        static_assert(kPairSlots == 4 && D >= 4, "the groups' slots; the ring is at least as deep");
        const uint32_t dst = tmem + lanes + kPairNT + 64u * grp;
        int next = grp, done = 0;                          // the group's next stage; units whose sums are drained
        int q = pair;                                      // the unit in hand
        float v[16][4];                                    // drained sums: runs of 16 tokens, 64 tokens apart
        int left = 0, c = 0;                               // runs still to be finished, and the first token of the next
        int m0 = 0, mv = 0, n = 0;                         // of the unit that they belong to: its rows of X, this thread's
                                                           // column, the column's scale and bias
        float sc = 0.0f, bi = 0.0f;
        bool turn = false;                                 // whether a run is next, or a stage
        while (ok) {
            const bool more = q < units && next < seq + stages, pending = seq > done * stages;
            if (left > 0 && (turn || !more)) {
                turn = false;
                --left;
                if (n < P.N && c < mv) {                   // (the residual is in L2: the copying warp asked for it)
                    // 16 rows at once, or eight with a residual, whose loads take as many registers: each form on its own
                    // nearly keeps within them (56 bytes of reloads in all; one form for both: 8 % more time, M 4096,
                    // N = K = 8192)
                    if (P.epi.residual) {
#pragma unroll
                        for (int h = 0; h < 16; h += 8) {
                            if (c + h >= mv) break;
                            float z[8];
#pragma unroll
                            for (int i = 0; i < 8; ++i) z[i] = v[(h + i) >> 2][i & 3];
                            lin_finish_as<true>(P.epi, z, mv - c - h, sc, bi, (int64_t)m0 + c + h, n);
                        }
                    } else {
                        float z[16];
#pragma unroll
                        for (int i = 0; i < 16; ++i) z[i] = v[i >> 2][i & 3];
                        lin_finish_as<false>(P.epi, z, mv - c, sc, bi, (int64_t)m0 + c, n);
                    }
                }
                c += 64;
                lin_move16(v, 0, 4);
                lin_move16(v, 4, 8);
                lin_move16(v, 8, 12);
                __syncwarp();
                continue;
            }
            // The sums of the unit before are drained when the MMAs have done their last stage, which is also when the last
            // of the four slots comes free: the group that waits for that slot drains first.
            if (pending && (!more || next - seq >= kPairSlots - 1)) {
                if (!g_wait_warp(acc_full, (uint32_t)done & 1u)) {
                    ok = false;
                    break;
                }
                ++done;
                asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
                lin_tmem_drain(tmem + lanes + 16u * grp, v);
                asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
                __syncwarp();
                if (lane == 0) lin_arrive_lead(acc_empty);
                c = 16 * grp;
                left = (mv - c + 63) >> 6;                 // (not positive where the unit has no token for the group)
                turn = next - seq >= kPairSlots;
                continue;
            }
            if (!more) {
                if (q >= units) break;
                const LinUnit u = lin_find<kPairNT>(P, q / rtps);
                m0 = u.m0;
                mv = u.m1 - u.m0;
                n = (2 * (q % rtps) + (int)rank) * kLinRows + r;
                if (n < P.N) {
                    sc = __half2float(__ushort_as_half(P.scale[(int64_t)u.e * P.N + n]));
                    bi = P.epi.bias ? lin_elem(P.epi.bias, (int64_t)u.e * P.N + n, P.epi.bias_bf16) : 0.0f;
                }
                seq += stages;
                q += pairs;
                continue;
            }
            // the slot first, as in linear_kernel
            const int s = next % D;
            if ((next >= kPairSlots && !g_wait_warp(tfree(grp), (uint32_t)(next / kPairSlots - 1) & 1u)) ||
                !g_wait_warp(full(s), (uint32_t)(next / D) & 1u)) {
                ok = false;
                break;
            }
            asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
            const uint32_t src = c_tile(s, 0) + 16u * r;
            lin_codes_to_tmem<QB>(src, dst);
            if (2 * (next - seq) + 1 < P.kbs) lin_codes_to_tmem<QB>(src + S::c_block, dst + 32u);
            asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
            asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
            __syncwarp();
            if (lane == 0) lin_arrive_lead(wready(grp));
            next += kPairSlots;
            turn = true;
        }
    }
    if (!ok && lane == 0 && P.status) atomicOr(reinterpret_cast<unsigned int*>(P.status), 0x4u);
    asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
    __syncwarp();
    lin_cluster_sync();                                    // nothing of this pair arrives on the other block any more
    if (warp == 1) {
        asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
    }
}

// K = 0: the sums are 0, the epilogue is all there is.  One block per row of Y.  With N = 0: a look at the offsets alone.
__global__ void __launch_bounds__(256) linear_empty_kernel(const __grid_constant__ LinParams P) {
    if (P.offsets && P.status && blockIdx.x == 0)
        for (int e = threadIdx.x; e < (int)P.E; e += blockDim.x) {
            const int p = P.offsets[e], q = P.offsets[e + 1];
            if (p < 0 || q < p || q > (int)P.M) atomicOr(reinterpret_cast<unsigned int*>(P.status), 0x8u);
        }
    if (P.N == 0) return;
    for (int64_t m = blockIdx.x; m < P.M; m += gridDim.x) {
        int64_t e = 0;
        if (P.offsets) {                                   // the expert of the row: the last that begins at or before it
            int64_t lo = 0, hi = P.E;
            while (hi - lo > 1) {
                const int64_t mid = (lo + hi) >> 1;
                if (P.offsets[mid] <= m) lo = mid;
                else hi = mid;
            }
            e = lo;
            if (m < P.offsets[e] || m >= P.offsets[e + 1]) continue;
        }
        for (int64_t n = threadIdx.x; n < P.N; n += blockDim.x) {
            float v[2] = {0.0f, 0.0f};
            lin_finish(P.epi, v, 1, 0.0f, P.epi.bias ? lin_elem(P.epi.bias, e * P.N + n, P.epi.bias_bf16) : 0.0f, m, n);
        }
    }
}

}  // namespace gq
