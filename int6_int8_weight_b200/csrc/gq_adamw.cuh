// gq_adamw.cuh -- one AdamW step over a batch of tensors, states in 32 or in
// 8 bits (the definition is in include/gq.h; every line of it is one binary32
// rounding).
//
// A step reads p, g, m, v and writes p, m, v once: 28 bytes per element with
// fp32 weights and states, 10 with bf16 weights and 8-bit states.  Bound with
// 32-bit states: HBM (the weights of 9 layers of d 512, 606 MB in all, in 93 us:
// 6.5 TB/s).  With 8-bit states the square root, the quotient,
// the fourth root and the hash come to 90 instructions an element, 104 with the
// first moment in square codes, and their issue is the bound: 16384 x 8192, fp32
// weights and bf16 gradients, in 451 us (4.2 TB/s), 506 with square codes, at 70 % of the
// issue slots.  48 registers (five blocks an SM) leave 36 bytes of spills.
//
// Split: a work item is a run of 2048 elements of one tensor (8 blocks of 256,
// one a warp), so that any list of tensors spreads evenly; a lane owns 8
// consecutive elements, which makes a block of 256 one warp: the block's
// maxima are two integer warp reductions and the new codes leave as one 8-byte
// store a lane.
#pragma once

#include "gq_device.cuh"

namespace gq {

constexpr int kAdamDesc = 200;            // tensors a launch (the parameter block stays below 32 KB)
constexpr int kAdamFew = 16;              // a batch of no more takes a small block: 18 KB of parameters cost the host time
constexpr int kAdamThreads = 256;
constexpr int kAdamItem = 8 * kAdamThreads;
constexpr float kAdamLow = 8.673617379884035e-19f, kAdamHigh = 1.152921504606847e18f;   // 2^-60, 2^60
constexpr float kAdamTiny = 8.271806125530277e-25f;   // 2^-80: blocks below it store 0

struct AdamDesc {
    void* p;
    const void* g;
    void* m;
    void* v;
    float* ms;
    float* vs;
    uint16_t* copy;
    int64_t numel;
    double wd;
    float decay;          // RN(1 - lr * wd)
    uint32_t key;         // of the hash, without the step
    int32_t flags;        // kAdam* bits
    int32_t pad;
};

constexpr int32_t kAdamPBf16 = 1, kAdamGBf16 = 2, kAdamVec = 4;

struct AdamStep {
    int32_t ndesc;
    uint32_t key_step;    // the step's share of the hash key
    double lr, beta1, beta2;
    double bias1;         // 1 - b1^t
    float b1, c1, b2, c2, eps;
    float inv_bc2;        // RN(1 / sqrt(1 - b2^t))
    float step_size;      // RN(lr / (1 - b1^t))
    float one;            // 1
    int32_t paired;       // eps is in the paired quotient's range: sqrt(v) inv_bc2 + eps is too
    const int64_t* d_step;
    const float* d_lr;
    const float* d_grad_scale;
};

template <int CAP>
struct AdamParams : AdamStep {
    int64_t start[CAP + 1];         // prefix sums of work items
    AdamDesc d[CAP];
};

constexpr uint32_t kAdamStepMul = 0x632BE5ABu, kAdamTensorMul = 0x2C1B3C6Du;

// 32 random bits of an element: two multiply-xorshift rounds over a seed that moves
// with the index by 2^32 / golden ratio (Knuth's multiplicative hashing).  The
// rounds' shifts and multipliers are a result of C. Wellons' published search for
// 32-bit mixers of low bias ("Prospecting for Hash Functions", 2018); the other
// constants only keep steps, tensors and high index words apart.
__device__ __forceinline__ uint32_t adam_seed(int64_t index, uint32_t key) {
    return (uint32_t)index * 0x9E3779B9u + (uint32_t)((uint64_t)index >> 32) * 0x7FEB3529u + key;
}
__device__ __forceinline__ uint32_t adam_mix(uint32_t z) {
    z = (z ^ (z >> 16)) * 0x21F0AAADu;
    z = (z ^ (z >> 15)) * 0x735A2D97u;
    return z ^ (z >> 15);
}

__device__ __forceinline__ float adam_root(float x) {
    float r;
    asm("sqrt.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

// Two elements in one register pair: a pair costs one instruction issue, which
// is what bounds the 8-bit step.  Every operation is one rounding.  The code
// generator fuses a paired product into a paired sum even where contraction is
// off, so a sum is written x * one + y with a 1 that it cannot see (a kernel
// parameter): a product times an unknown number has nothing to be fused with.
using AdamF2 = uint64_t;
__device__ __forceinline__ AdamF2 adam2(float lo, float hi) {
    AdamF2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
    return r;
}
__device__ __forceinline__ AdamF2 adam2(float x) { return adam2(x, x); }
__device__ __forceinline__ void adam2_out(AdamF2 a, float& lo, float& hi) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(a));
}
__device__ __forceinline__ AdamF2 adam2_fma(AdamF2 a, AdamF2 b, AdamF2 c) {
    AdamF2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ AdamF2 adam2_mul(AdamF2 a, AdamF2 b) { return adam2_fma(a, b, adam2(-0.0f)); }
struct AdamOne {
    AdamF2 one, minus;           // (1, 1) and (-1, -1)
    __device__ __forceinline__ AdamF2 add(AdamF2 a, AdamF2 b) const { return adam2_fma(a, one, b); }
    __device__ __forceinline__ AdamF2 sub(AdamF2 a, AdamF2 b) const { return adam2_fma(b, minus, a); }
    __device__ __forceinline__ AdamF2 add_down(AdamF2 a, AdamF2 b) const {   // rounded down
        AdamF2 r;
        asm("fma.rm.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(one), "l"(b));
        return r;
    }
};
// Square root and quotient of pairs, correctly rounded, by Newton steps on the
// special function unit's estimates with exact residuals (Markstein): for the
// root r of v, v - r^2 decides the last bit; for the quotient q of m and d,
// m - d q, times a correctly rounded reciprocal.  The residuals are exact, and
// so the results those of the IEEE operations, while nothing under- or
// overflows: 2^-60 <= v <= 2^60, 2^-60 <= |d| <= 2^60, 2^-60 <= |m| <= 2^60.
// (Checked against the IEEE operations for every significand of v with both
// parities of the exponent, every significand of d's reciprocal, and 2^33
// quotients.)  11 instructions for an element against 22 for the IEEE operations,
// which test every operand by themselves.
__device__ __forceinline__ AdamF2 adam2_sqrt(AdamF2 v) {
    float v0, v1, y0, y1;
    adam2_out(v, v0, v1);
    asm("rsqrt.approx.ftz.f32 %0, %1;" : "=f"(y0) : "f"(v0));
    asm("rsqrt.approx.ftz.f32 %0, %1;" : "=f"(y1) : "f"(v1));
    const AdamF2 y = adam2(y0, y1), g = adam2_mul(v, y), h = adam2_mul(y, adam2(-0.5f));   // v^(1/2), -v^(-1/2) / 2
    const AdamF2 e = adam2_fma(g, h, adam2(0.5f));
    const AdamF2 g1 = adam2_fma(g, e, g), h1 = adam2_fma(h, e, h);
    return adam2_fma(adam2_fma(g1, g1, adam2_mul(v, adam2(-1.0f))), h1, g1);
}
__device__ __forceinline__ AdamF2 adam2_div(AdamF2 m, AdamF2 d) {
    float d0, d1, y0, y1;
    adam2_out(d, d0, d1);
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y0) : "f"(d0));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y1) : "f"(d1));
    const AdamF2 nd = adam2_mul(d, adam2(-1.0f)), y = adam2(y0, y1);
    const AdamF2 r = adam2_fma(y, adam2_fma(nd, y, adam2(1.0f)), y);    // RN(1 / d)
    const AdamF2 q = adam2_mul(m, r), q1 = adam2_fma(adam2_fma(nd, q, m), r, q);
    return adam2_fma(adam2_fma(nd, q1, m), r, q1);
}

// f(q) = RN((q^2)^2); q^2 is exact.
__device__ __forceinline__ AdamF2 adam2_fourth(AdamF2 q) {
    const AdamF2 t = adam2_mul(q, q);
    return adam2_mul(t, t);
}

// 8 consecutive elements of a float / bf16 array as floats (vector path:
// 16-byte aligned and all in range; else element by element, 0 past n).
__device__ __forceinline__ void adam_load(float (&x)[8], const void* base, int64_t e, int n, bool bf16, bool vec) {
    if (bf16) {
        const uint16_t* s = static_cast<const uint16_t*>(base) + e;
        if (vec) {
            const uint4 u = __ldcs(reinterpret_cast<const uint4*>(s));
            const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                x[2 * i] = __uint_as_float(w[i] << 16);
                x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
            }
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) x[i] = i < n ? bf16_bits_to_float(s[i]) : 0.0f;
        }
    } else {
        const float* s = static_cast<const float*>(base) + e;
        if (vec) {
            const float4 a = __ldcs(reinterpret_cast<const float4*>(s));
            const float4 b = __ldcs(reinterpret_cast<const float4*>(s) + 1);
            x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
            x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) x[i] = i < n ? s[i] : 0.0f;
        }
    }
}

__device__ __forceinline__ void adam_store(const float (&x)[8], void* base, int64_t e, int n, bool bf16, bool vec) {
    if (bf16) {
        uint16_t* s = static_cast<uint16_t*>(base) + e;
        if (vec) {
            uint32_t w[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
                w[i] = *reinterpret_cast<const uint32_t*>(&h);
            }
            __stcs(reinterpret_cast<uint4*>(s), make_uint4(w[0], w[1], w[2], w[3]));
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (i < n) s[i] = float_to_bf16_bits(x[i]);
        }
    } else {
        float* s = static_cast<float*>(base) + e;
        if (vec) {
            __stcs(reinterpret_cast<float4*>(s), make_float4(x[0], x[1], x[2], x[3]));
            __stcs(reinterpret_cast<float4*>(s) + 1, make_float4(x[4], x[5], x[6], x[7]));
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (i < n) s[i] = x[i];
        }
    }
}

__device__ __forceinline__ void adam_load8(uint32_t (&c)[2], const void* base, int64_t e, int n, bool vec) {
    const uint8_t* s = static_cast<const uint8_t*>(base) + e;
    if (vec) {
        const uint2 u = __ldcs(reinterpret_cast<const uint2*>(s));
        c[0] = u.x;
        c[1] = u.y;
    } else {
        c[0] = c[1] = 0u;
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < n) c[i >> 2] |= (uint32_t)s[i] << (8 * (i & 3));
    }
}

__device__ __forceinline__ void adam_store8(const uint32_t (&c)[2], void* base, int64_t e, int n, bool vec) {
    uint8_t* s = static_cast<uint8_t*>(base) + e;
    if (vec) {
        __stcs(reinterpret_cast<uint2*>(s), make_uint2(c[0], c[1]));
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < n) s[i] = (uint8_t)(c[i >> 2] >> (8 * (i & 3)));
    }
}

// What the launch's tensors hold as states: 32 bits, or 8 with the first moment in linear or in square codes.
enum AdamState { kAdam32, kAdam8Linear, kAdam8Square };

template <int ST, int CAP>
__global__ void __launch_bounds__(kAdamThreads, ST == kAdam32 ? 4 : 5)
    adamw_kernel(const __grid_constant__ AdamParams<CAP> P) {
    constexpr bool S8 = ST != kAdam32;
    __shared__ float s_step[3];
    float inv_bc2 = P.inv_bc2, step_size = P.step_size;
    double lr = P.lr;
    uint32_t key_step = P.key_step;
    if (P.d_step || P.d_lr) {
        // the step's scalars from device memory (a captured step): binary64, as on the host
        if (threadIdx.x == 0) {
            if (P.d_lr) lr = (double)*P.d_lr;
            if (P.d_step) {
                const int64_t t = *P.d_step;
                key_step = (uint32_t)t * kAdamStepMul;
                inv_bc2 = (float)(1.0 / sqrt(1.0 - pow(P.beta2, (double)t)));
                step_size = (float)(lr / (1.0 - pow(P.beta1, (double)t)));
            } else {
                step_size = (float)(lr / P.bias1);
            }
            s_step[0] = inv_bc2;
            s_step[1] = step_size;
            s_step[2] = __uint_as_float(key_step);
        }
        __syncthreads();
        inv_bc2 = s_step[0];
        step_size = s_step[1];
        key_step = __float_as_uint(s_step[2]);
        if (P.d_lr) lr = (double)*P.d_lr;
    }
    const AdamOne U{adam2(P.one), adam2(-P.one)};
    const float gs = P.d_grad_scale ? *P.d_grad_scale : 1.0f;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t total = P.start[P.ndesc];
    for (int64_t item = blockIdx.x; item < total; item += gridDim.x) {
        int lo = 0, hi = P.ndesc;                          // the descriptor that owns the item
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (P.start[mid] <= item) lo = mid;
            else hi = mid;
        }
        const AdamDesc& D = P.d[lo];
        const int64_t blk = (item - P.start[lo]) * (kAdamItem / 256) + warp;   // block of 256 of the tensor
        const int64_t e = blk * 256 + 8 * lane;
        if (blk * 256 >= D.numel) continue;                // a whole warp: its block is past the end
        const int n = (int)max((int64_t)0, min((int64_t)8, D.numel - e));
        const bool vec = (D.flags & kAdamVec) && n == 8;
        const bool pb = D.flags & kAdamPBf16, gb = D.flags & kAdamGBf16;
        const float decay = P.d_lr ? (float)(1.0 - lr * D.wd) : D.decay;
        float p[8], g[8], m[8], v[8];
        adam_load(g, D.g, e, n, gb, vec);
        adam_load(p, D.p, e, n, pb, vec);
        if constexpr (S8) {
            uint32_t cm[2], cv[2];
            adam_load8(cm, D.m, e, n, vec);
            adam_load8(cv, D.v, e, n, vec);
            const float ms = D.ms[blk], vs = D.vs[blk];
            // a byte under the exponent of 2^23 less 2^23 is its value, exactly (the signed one offset by 128)
            auto bytes = [&](uint32_t c, int i) {
                return adam2(__uint_as_float(__byte_perm(c, 0x4B000000u, 0x7440 + i)),
                             __uint_as_float(__byte_perm(c, 0x4B000000u, 0x7441 + i)));
            };
#pragma unroll
            for (int i = 0; i < 8; i += 2) {
                const AdamF2 qm = U.add(bytes(cm[i >> 2] ^ 0x80808080u, i & 3), adam2(-8388736.0f));
                const AdamF2 qv = U.add(bytes(cv[i >> 2], i & 3), adam2(-8388608.0f));
                if constexpr (ST == kAdam8Square) {
                    float q0, q1;
                    adam2_out(qm, q0, q1);
                    adam2_out(adam2_mul(adam2_mul(qm, adam2(fabsf(q0), fabsf(q1))), adam2(ms)), m[i], m[i + 1]);
                } else {
                    adam2_out(adam2_mul(qm, adam2(ms)), m[i], m[i + 1]);
                }
                adam2_out(adam2_mul(adam2_fourth(qv), adam2(vs)), v[i], v[i + 1]);
            }
        } else {
            adam_load(m, D.m, e, n, false, vec);
            adam_load(v, D.v, e, n, false, vec);
        }
#pragma unroll
        for (int i = 0; i < 8; i += 2) {
            AdamF2 g2 = adam2(g[i], g[i + 1]);
            if (P.d_grad_scale) g2 = adam2_mul(g2, adam2(gs));
            const AdamF2 m2 = U.add(adam2_mul(adam2(m[i], m[i + 1]), adam2(P.b1)), adam2_mul(g2, adam2(P.c1)));
            const AdamF2 v2 = U.add(adam2_mul(adam2(v[i], v[i + 1]), adam2(P.b2)),
                                    adam2_mul(adam2_mul(g2, g2), adam2(P.c2)));
            adam2_out(m2, m[i], m[i + 1]);
            adam2_out(v2, v[i], v[i + 1]);
        }
        // p' = p decay - (m / (sqrt(v) inv_bc2 + eps)) step_size.  32-bit states wait for memory and take the IEEE
        // operations; so do lanes whose values leave the range of the paired ones.
        float am = 0.0f, av = 0.0f;                        // (past the tensor's end m and v are 0)
        bool plain = !S8;
        if constexpr (S8) {
            float lo_m = fabsf(m[0]), lo_v = v[0];
            am = lo_m;
            av = lo_v;
#pragma unroll
            for (int i = 1; i < 8; ++i) {
                lo_m = fminf(lo_m, fabsf(m[i]));
                lo_v = fminf(lo_v, v[i]);
                am = fmaxf(am, fabsf(m[i]));
                av = fmaxf(av, v[i]);
            }
            // (a NaN, which min and max pass over, comes out of either form as a NaN)
            plain = !(fminf(lo_m, lo_v) >= kAdamLow && fmaxf(am, av) <= kAdamHigh) || !P.paired;
        }
#pragma unroll
        for (int i = 0; i < 8; i += 2) {
            AdamF2 u2;
            if (plain) {
                const AdamF2 r2 = adam2(__fsqrt_rn(v[i]), __fsqrt_rn(v[i + 1]));
                float d0, d1;
                adam2_out(U.add(adam2_mul(r2, adam2(inv_bc2)), adam2(P.eps)), d0, d1);
                u2 = adam2(__fdiv_rn(m[i], d0), __fdiv_rn(m[i + 1], d1));
            } else {
                u2 = adam2_div(adam2(m[i], m[i + 1]), U.add(adam2_mul(adam2_sqrt(adam2(v[i], v[i + 1])), adam2(inv_bc2)),
                                                            adam2(P.eps)));
            }
            adam2_out(U.sub(adam2_mul(adam2(p[i], p[i + 1]), adam2(decay)), adam2_mul(u2, adam2(step_size))), p[i], p[i + 1]);
        }
        adam_store(p, D.p, e, n, pb, vec);
        if (D.copy) adam_store(p, D.copy, e, n, true, vec);
        if constexpr (!S8) {
            adam_store(m, D.m, e, n, false, vec);
            adam_store(v, D.v, e, n, false, vec);
            continue;
        }
        am = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(am)));   // non-negative: ordered like their bits
        av = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(av)));
        const bool km = am >= kAdamTiny, kv = av >= kAdamTiny;
        const float im = km ? __fdiv_rn(ST == kAdam8Square ? 16129.0f : 127.0f, am) : 0.0f;   // 127^2
        const float iv = kv ? __fdiv_rn(4228250625.0f, av) : 0.0f;   // 255^4
        uint32_t cm[2] = {0u, 0u}, cv[2] = {0u, 0u};
        const uint32_t z0 = adam_seed(e, D.key + key_step);
#pragma unroll
        for (int i = 0; i < 8; i += 2) {
            // e is a multiple of 8: no carry into the index's high word
            const uint32_t za = adam_mix(z0 + (uint32_t)i * 0x9E3779B9u), zb = adam_mix(z0 + (uint32_t)(i + 1) * 0x9E3779B9u);
            // 16 bits k under the exponent of 2^23: (2^23 + k) * 2^-16 - 2^7 = k * 2^-16, exactly
            auto unit = [](uint32_t a, uint32_t b, uint32_t half) {
                return adam2_fma(adam2(__uint_as_float(__byte_perm(a, 0x4B000000u, half)),
                                       __uint_as_float(__byte_perm(b, 0x4B000000u, half))),
                                 adam2(1.52587890625e-5f), adam2(-128.0f));
            };
            const AdamF2 um = unit(za, zb, 0x7432), uv = unit(za, zb, 0x7410);
            float t0, t1;
            if constexpr (ST == kAdam8Square) {
                // |q| = q0 + (u (2 q0 + 1) < x - q0^2): q0 as the fourth root's below, from one root; 16 + 8 bits of
                // u (2 q0 + 1) are exact.  The sum with kMagic holds the signed code in its low byte.
                const AdamF2 x = adam2_mul(adam2(fabsf(m[i]), fabsf(m[i + 1])), adam2(im));
                float x0, x1, q0, q1, f0, f1;
                adam2_out(x, x0, x1);
                adam2_out(adam2_mul(adam2(adam_root(x0), adam_root(x1)), adam2(1.000003814697265625f)), q0, q1);
                AdamF2 q = U.add(U.add_down(adam2(fminf(q0, 126.0f), fminf(q1, 126.0f)), adam2(8388608.0f)),
                                 adam2(-8388608.0f));
                AdamF2 f = adam2_mul(q, q);
                adam2_out(f, f0, f1);
                if (f0 > x0 || f1 > x1) {
                    adam2_out(q, q0, q1);
                    q = adam2(f0 > x0 ? q0 - 1.0f : q0, f1 > x1 ? q1 - 1.0f : q1);
                    f = adam2_mul(q, q);
                }
                float s0, s1, r0, r1;
                adam2_out(adam2_mul(um, adam2_fma(q, adam2(2.0f), U.one)), s0, s1);
                adam2_out(U.sub(x, f), r0, r1);
                adam2_out(U.add(q, adam2(s0 < r0 ? 1.0f : 0.0f, s1 < r1 ? 1.0f : 0.0f)), q0, q1);
                adam2_out(U.add(adam2(copysignf(q0, m[i]), copysignf(q1, m[i + 1])), adam2(kMagic)), t0, t1);
            } else {
                // floor by an addition rounded down: the code is in the low byte of the sum's bits (it is at most 127:
                // m' * RN(127 / a) is below 127 + 2^-15, and u at most 1 - 2^-16)
                adam2_out(U.add(adam2_mul(adam2(m[i], m[i + 1]), adam2(im)), um), t0, t1);
                adam2_out(U.add_down(adam2(fmaxf(t0, -127.0f), fmaxf(t1, -127.0f)), adam2(kMagic)), t0, t1);
            }
            const AdamF2 x = adam2_mul(adam2(v[i], v[i + 1]), adam2(iv));
            float x0, x1, q0, q1, f0, f1;
            adam2_out(x, x0, x1);
            // q0: a fourth root good to 2^-20, raised by 2^-18, so that its floor is never too small and at most one too
            // large; set right against f itself.  qi = q + 2^23: the code in the low byte.
            adam2_out(adam2_mul(adam2(adam_root(adam_root(x0)), adam_root(adam_root(x1))), adam2(1.000003814697265625f)),
                      q0, q1);
            AdamF2 qi = U.add_down(adam2(fminf(q0, 254.0f), fminf(q1, 254.0f)), adam2(8388608.0f));
            AdamF2 q = U.add(qi, adam2(-8388608.0f));
            AdamF2 f = adam2_fourth(q);
            adam2_out(f, f0, f1);
            if (f0 > x0 || f1 > x1) {
                adam2_out(q, q0, q1);
                q = adam2(f0 > x0 ? q0 - 1.0f : q0, f1 > x1 ? q1 - 1.0f : q1);
                qi = U.add(q, adam2(8388608.0f));
                f = adam2_fourth(q);
            }
            // one more where u (f(q + 1) - f(q)) < x - f(q); at q = 0 where 0 < x
            float s0, s1, r0, r1;
            adam2_out(q, q0, q1);
            adam2_out(adam2_mul(adam2_mul(uv, U.sub(adam2_fourth(U.add(q, U.one)), f)),
                                adam2(fminf(q0, 1.0f), fminf(q1, 1.0f))), s0, s1);
            adam2_out(U.sub(x, f), r0, r1);
            adam2_out(U.add(qi, adam2(s0 < r0 ? 1.0f : 0.0f, s1 < r1 ? 1.0f : 0.0f)), q0, q1);
            // two code bytes into their word
            const uint32_t sel = (i & 2) ? 0x5410u : 0x3254u;
            cm[i >> 2] = __byte_perm(cm[i >> 2], __byte_perm(__float_as_uint(t0), __float_as_uint(t1), 0x0040), sel);
            cv[i >> 2] = __byte_perm(cv[i >> 2], __byte_perm(__float_as_uint(q0), __float_as_uint(q1), 0x0040), sel);
        }
        adam_store8(cm, D.m, e, n, vec);
        adam_store8(cv, D.v, e, n, vec);
        if (lane == 0) {
            // RN(1 / 127), RN(1 / 127^2)
            D.ms[blk] = km ? __fmul_rn(am, ST == kAdam8Square ? 6.200012400024800e-05f : 0.007874015748031496f) : 0.0f;
            D.vs[blk] = kv ? __fmul_rn(av, 2.3650442906278766e-10f) : 0.0f;     // RN(1 / 255^4)
        }
    }
}

}  // namespace gq
