// gq_adamw.cuh -- one AdamW step over a batch of tensors, states in 32 or in
// 8 bits (the definition is in include/gq.h; every line of it is one binary32
// rounding).
//
// Bound: HBM.  A step reads p, g, m, v and writes p, m, v once: 28 bytes per
// element with fp32 weights and states, 10 with bf16 weights and 8-bit states.
// The arithmetic (one IEEE square root and one IEEE division an element, and
// for 8-bit states two fourth roots' worth of comparisons and a hash) is about
// 60 / 110 instructions an element.
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
constexpr int kAdamThreads = 256;
constexpr int kAdamItem = 8 * kAdamThreads;
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

struct AdamParams {
    int32_t ndesc;
    uint32_t key_step;    // the step's share of the hash key
    double lr, beta1, beta2;
    double bias1;         // 1 - b1^t
    float b1, c1, b2, c2, eps;
    float inv_bc2;        // RN(1 / sqrt(1 - b2^t))
    float step_size;      // RN(lr / (1 - b1^t))
    const int64_t* d_step;
    const float* d_lr;
    const float* d_grad_scale;
    int64_t start[kAdamDesc + 1];   // prefix sums of work items
    AdamDesc d[kAdamDesc];
};

constexpr uint32_t kAdamStepMul = 0x632BE5ABu, kAdamTensorMul = 0x2C1B3C6Du;

// 32 random bits of an element: two multiply-xorshift rounds over a seed that
// moves by a constant with the index.
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
    asm("sqrt.approx.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

// f(q) = RN((q^2)^2); q^2 is exact.
__device__ __forceinline__ float adam_fourth(float q) {
    const float t = __fmul_rn(q, q);
    return __fmul_rn(t, t);
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

// S8: the launch's tensors have 8-bit states.
template <bool S8>
__global__ void __launch_bounds__(kAdamThreads, 4) adamw_kernel(const __grid_constant__ AdamParams P) {
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
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                // a byte under the exponent of 2^23 less 2^23 is its value, exactly (the signed one offset by 128)
                const uint32_t bm = __byte_perm(cm[i >> 2] ^ 0x80808080u, 0x4B000000u, 0x7440 + (i & 3));
                const uint32_t bv = __byte_perm(cv[i >> 2], 0x4B000000u, 0x7440 + (i & 3));
                m[i] = __fmul_rn(__fsub_rn(__uint_as_float(bm), 8388736.0f), ms);
                v[i] = __fmul_rn(adam_fourth(__fsub_rn(__uint_as_float(bv), 8388608.0f)), vs);
            }
        } else {
            adam_load(m, D.m, e, n, false, vec);
            adam_load(v, D.v, e, n, false, vec);
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float gi = P.d_grad_scale ? __fmul_rn(g[i], gs) : g[i];
            m[i] = __fadd_rn(__fmul_rn(m[i], P.b1), __fmul_rn(gi, P.c1));
            v[i] = __fadd_rn(__fmul_rn(v[i], P.b2), __fmul_rn(__fmul_rn(gi, gi), P.c2));
            const float d = __fadd_rn(__fmul_rn(__fsqrt_rn(v[i]), inv_bc2), P.eps);
            const float u = __fmul_rn(__fdiv_rn(m[i], d), step_size);
            p[i] = __fsub_rn(__fmul_rn(p[i], decay), u);
        }
        adam_store(p, D.p, e, n, pb, vec);
        if (D.copy) adam_store(p, D.copy, e, n, true, vec);
        if constexpr (!S8) {
            adam_store(m, D.m, e, n, false, vec);
            adam_store(v, D.v, e, n, false, vec);
            continue;
        }
        // past the tensor's end m and v are 0: they do not raise the maxima
        float am = 0.0f, av = 0.0f;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            if (i >= n) m[i] = v[i] = 0.0f;
            am = fmaxf(am, fabsf(m[i]));
            av = fmaxf(av, v[i]);
        }
        am = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(am)));   // non-negative: ordered like their bits
        av = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(av)));
        const bool km = am >= kAdamTiny, kv = av >= kAdamTiny;
        const float im = km ? __fdiv_rn(127.0f, am) : 0.0f;
        const float iv = kv ? __fdiv_rn(4228250625.0f, av) : 0.0f;   // 255^4
        uint32_t cm[2] = {0u, 0u}, cv[2] = {0u, 0u};
        const uint32_t z0 = adam_seed(e, D.key + key_step);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const uint32_t z = adam_mix(z0 + (uint32_t)i * 0x9E3779B9u);   // e is a multiple of 8: no carry into its high word
            // 16 bits k under the exponent of 1 less 1: k * 2^-16, exactly
            const float um = __fsub_rn(__uint_as_float((z >> 9 & 0x007FFF80u) | 0x3F800000u), 1.0f);
            const float uv = __fsub_rn(__uint_as_float((z << 7 & 0x007FFF80u) | 0x3F800000u), 1.0f);
            // floor by an addition rounded down: the code is in the low byte of the sum's bits
            const float tm = fminf(fmaxf(__fadd_rn(__fmul_rn(m[i], im), um), -127.0f), 127.0f);
            const uint32_t qm = __float_as_uint(__fadd_rd(tm, kMagic));
            const float x = __fmul_rn(v[i], iv);
            // q0: an approximate fourth root, at most one off, set right against f itself
            float q0 = __fsub_rn(__fadd_rd(fminf(adam_root(adam_root(x)), 254.0f), 8388608.0f), 8388608.0f);
            float f0 = adam_fourth(q0), f1 = adam_fourth(q0 + 1.0f);
            if (f0 > x) {
                q0 -= 1.0f;
                f1 = f0;
                f0 = adam_fourth(q0);
            } else if (f1 <= x && q0 < 254.0f) {
                q0 += 1.0f;
                f0 = f1;
                f1 = adam_fourth(q0 + 1.0f);
            }
            float qv = __fmul_rn(uv, __fsub_rn(f1, f0)) < __fsub_rn(x, f0) ? q0 + 1.0f : q0;
            if (x > 0.0f) qv = fmaxf(qv, 1.0f);
            const uint32_t bv = __float_as_uint(__fadd_rn(qv, 8388608.0f));
            const uint32_t sel = (i & 3) == 0 ? 0x3214 : (i & 3) == 1 ? 0x3240 : (i & 3) == 2 ? 0x3410 : 0x4210;
            cm[i >> 2] = __byte_perm(cm[i >> 2], qm, sel);
            cv[i >> 2] = __byte_perm(cv[i >> 2], bv, sel);
        }
        adam_store8(cm, D.m, e, n, vec);
        adam_store8(cv, D.v, e, n, vec);
        if (lane == 0) {
            D.ms[blk] = km ? __fmul_rn(am, 0.007874015748031496f) : 0.0f;       // RN(1 / 127)
            D.vs[blk] = kv ? __fmul_rn(av, 2.3650442906278766e-10f) : 0.0f;     // RN(1 / 255^4)
        }
    }
}

}  // namespace gq
