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
// the tile out.  Bound: HBM, once per weight; the packed rows may start at any
// byte, so they are read byte by byte (through L1).
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

__device__ __forceinline__ uint32_t lin_sub2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

// The 8 pairs of codes of one int6 group (three words) as bf16x2 integers.  A
// 6-bit field u in a half's low bits under 0x4300 is the bf16 number 128 + u; less
// 160 it is q, exactly.
__device__ __forceinline__ void lin_codes6(uint32_t w0, uint32_t w1, uint32_t w2, uint32_t (&o)[8]) {
    constexpr uint32_t m = 0x003F003Fu, h = 0x43004300u, s = 0x43204320u;
    o[0] = lin_sub2((w0 & m) | h, s);
    o[1] = lin_sub2((w1 & m) | h, s);
    o[2] = lin_sub2((w2 & m) | h, s);
    o[3] = lin_sub2((w0 >> 6 & m) | h, s);
    o[4] = lin_sub2((w1 >> 6 & m) | h, s);
    o[5] = lin_sub2((w2 >> 6 & m) | h, s);
    o[6] = lin_sub2((w0 >> 12 & 0x000F000Fu) | ((w2 >> 8 & 0x00300030u) | h), s);
    o[7] = lin_sub2((w1 >> 12 & 0x000F000Fu) | ((w2 >> 10 & 0x00300030u) | h), s);
}

// The two pairs of an int8 word: the low seven bits give 128 + low, the sign bit
// under 0x4300 is 128 or 256, and their difference is q, exactly.
__device__ __forceinline__ void lin_codes8(uint32_t w, uint32_t& a, uint32_t& b) {
    constexpr uint32_t m = 0x007F007Fu, t = 0x00800080u, h = 0x43004300u;
    const uint32_t v = w >> 8;
    a = lin_sub2((w & m) | h, (w & t) | h);
    b = lin_sub2((v & m) | h, (v & t) | h);
}

// -------------------------------------------------------------- epilogue --

struct LinEpi {
    const void* bias;            // [N] (grouped: [E, N]) or null
    const void* residual;        // [M, ldr] or null
    void* y;                     // [M, ldy]
    int64_t ldr, ldy;
    int32_t bias_bf16, residual_bf16, y_bf16, act;
};

__device__ __forceinline__ float lin_act(float z, int act) {
    switch (act) {
        case GQ_ACT_RELU: return z < 0.0f ? 0.0f : z;      // NaN stays
        case GQ_ACT_RELU2: z = z < 0.0f ? 0.0f : z; return z * z;
        case GQ_ACT_LEAKY_RELU2: z = z < 0.0f ? 0.5f * z : z; return z * z;
        case GQ_ACT_SILU: return z / (1.0f + expf(-z));
        case GQ_ACT_GELU: return 0.5f * z * (1.0f + erff(z * 0.70710678118654752f));
        case GQ_ACT_GELU_TANH: return 0.5f * z * (1.0f + tanhf(0.79788456080286536f * (z + 0.044715f * z * z * z)));
        default: return z;
    }
}

__device__ __forceinline__ float lin_elem(const void* p, int64_t i, int bf16) {
    return bf16 ? bf16_bits_to_float(static_cast<const uint16_t*>(p)[i]) : static_cast<const float*>(p)[i];
}

// Y[m, n] from the sum, the row's scale and bias.
__device__ __forceinline__ void lin_finish(const LinEpi& E, float acc, float s, float b, int64_t m, int64_t n) {
    float z = acc * s;
    if (E.bias) z += b;
    float y = lin_act(z, E.act);
    if (E.residual) y += lin_elem(E.residual, m * E.ldr + n, E.residual_bf16);
    if (E.y_bf16) static_cast<uint16_t*>(E.y)[m * E.ldy + n] = float_to_bf16_bits(y);
    else static_cast<float*>(E.y)[m * E.ldy + n] = y;
}

struct LinParams {
    const uint16_t* x;
    const uint8_t* tiles;
    const uint16_t* scale;
    const int32_t* offsets;      // [E + 1] or null (one weight)
    int32_t* status;
    int64_t M, N, K, ldx, kbs, rts, E;
    LinEpi epi;
};

// The rows [a, b) of expert e within [0, M), and whether its offsets are right.
__device__ __forceinline__ bool lin_rows(const int32_t* off, int64_t e, int64_t M, int64_t& a, int64_t& b) {
    const int32_t p = off[e], q = off[e + 1];
    a = max((int64_t)p, (int64_t)0);
    b = min((int64_t)q, M);
    return p >= 0 && q >= p && q <= M;
}

// The plainest form: one thread per row of a tile, 8 tokens at a time.
template <int QB>
__global__ void __launch_bounds__(kLinRows) linear_kernel(const __grid_constant__ LinParams P) {
    __shared__ float xs[8][kLinK];
    const int r = threadIdx.x;
    const int64_t rt = blockIdx.x, e = blockIdx.z;
    int64_t a = 0, b = P.M;
    if (P.offsets && !lin_rows(P.offsets, e, P.M, a, b)) {
        if (P.status && r == 0) atomicOr(reinterpret_cast<unsigned int*>(P.status), 8u);
        return;
    }
    const int64_t n = rt * kLinRows + r;
    const uint8_t* tile = P.tiles + (e * P.rts + rt) * P.kbs * lin_block_bytes(QB);
    const float s = n < P.N ? __half2float(__ushort_as_half(P.scale[e * P.N + n])) : 0.0f;
    const float bias = P.epi.bias && n < P.N ? lin_elem(P.epi.bias, e * P.N + n, P.epi.bias_bf16) : 0.0f;
    for (int64_t m0 = a + 8 * blockIdx.y; m0 < b; m0 += 8 * gridDim.y) {
        float acc[8] = {};
        for (int64_t kb = 0; kb < P.kbs; ++kb) {
            __syncthreads();
            for (int i = r; i < 8 * kLinK; i += kLinRows) {
                const int64_t m = m0 + i / kLinK, k = kb * kLinK + i % kLinK;
                xs[i / kLinK][i % kLinK] = m < b && k < P.K ? bf16_bits_to_float(P.x[m * P.ldx + k]) : 0.0f;
            }
            __syncthreads();
            const uint4* src = reinterpret_cast<const uint4*>(tile + kb * lin_block_bytes(QB)) + r;
            uint32_t w[16], o[32];
#pragma unroll
            for (int c = 0; c < (QB == 6 ? 3 : 4); ++c) {
                const uint4 u = src[c * kLinRows];
                w[4 * c] = u.x; w[4 * c + 1] = u.y; w[4 * c + 2] = u.z; w[4 * c + 3] = u.w;
            }
            if constexpr (QB == 6) {
#pragma unroll
                for (int g = 0; g < 4; ++g) {
                    uint32_t t[8];
                    lin_codes6(w[3 * g], w[3 * g + 1], w[3 * g + 2], t);
#pragma unroll
                    for (int j = 0; j < 8; ++j) o[8 * g + j] = t[j];
                }
            } else {
#pragma unroll
                for (int j = 0; j < 16; ++j) lin_codes8(w[j], o[2 * j], o[2 * j + 1]);
            }
#pragma unroll
            for (int i = 0; i < kLinK; ++i) {
                const float q = (i & 1) ? __uint_as_float(o[i >> 1] & 0xFFFF0000u) : __uint_as_float(o[i >> 1] << 16);
#pragma unroll
                for (int t = 0; t < 8; ++t) acc[t] += xs[t][i] * q;
            }
        }
        if (n < P.N)
            for (int t = 0; t < 8; ++t)
                if (m0 + t < b) lin_finish(P.epi, acc[t], s, bias, m0 + t, n);
    }
}

}  // namespace gq
