// gq_adamw.cu -- host side of gq_adamw_step (include/gq.h).
#include <algorithm>
#include <cmath>
#include <cstring>

#include "gq_adamw.cuh"
#include "gq_host.h"

namespace {

using namespace gq;

static_assert(sizeof(gq_adamw_tensor) == 88 && sizeof(gq_adamw_hyper) == 72,
              "the layouts are part of the ABI (the Python binding mirrors them)");
static_assert(sizeof(AdamParams<kAdamDesc>) <= 32764, "kernel parameters end at 32764 bytes");

// The states of a tensor, -1 where state_bits is none of them.
int adam_state(const gq_adamw_tensor& t) {
    return t.state_bits == 32 ? kAdam32 : t.state_bits == 8 ? kAdam8Linear
         : t.state_bits == GQ_ADAMW_8_SQUARE ? kAdam8Square : -1;
}

gq_status check_adamw(const gq_adamw_tensor& t) {
    if (t.reserved != 0 || t.numel < 0) return GQ_ERR_INVALID_ARG;
    if ((t.p_dtype != GQ_F32 && t.p_dtype != GQ_BF16) || (t.g_dtype != GQ_F32 && t.g_dtype != GQ_BF16))
        return GQ_ERR_INVALID_ARG;
    if (adam_state(t) < 0) return GQ_ERR_INVALID_ARG;
    const bool s8 = t.state_bits != 32;
    if (!std::isfinite(t.weight_decay)) return GQ_ERR_INVALID_ARG;
    if (t.numel > INT64_MAX / 16) return GQ_ERR_INVALID_ARG;
    if (t.numel == 0) return GQ_OK;
    if (!t.p || !t.g || !t.m || !t.v) return GQ_ERR_INVALID_ARG;
    if (s8 ? (!t.m_scale || !t.v_scale) : (t.m_scale || t.v_scale)) return GQ_ERR_INVALID_ARG;
    const size_t ps = t.p_dtype == GQ_F32 ? 4 : 2, gs = t.g_dtype == GQ_F32 ? 4 : 2, ss = s8 ? 1 : 4;
    if (!aligned(t.p, ps) || !aligned(t.g, gs) || !aligned(t.m, ss) || !aligned(t.v, ss) ||
        (t.p_copy && !aligned(t.p_copy, 2)) || (t.m_scale && (!aligned(t.m_scale, 4) || !aligned(t.v_scale, 4))))
        return GQ_ERR_MISALIGNED;
    return GQ_OK;
}

// The launches of a step; S holds all that does not depend on the tensors.
template <int CAP>
gq_status launch_adamw(const gq_adamw_tensor* t, int n, const gq_adamw_hyper* h, const AdamStep& S, cudaStream_t stream) {
    AdamParams<CAP> P;
    static_cast<AdamStep&>(P) = S;
    // the tensors of each kind of states, up to CAP a launch
    for (const int state : {kAdam32, kAdam8Linear, kAdam8Square}) {
        const bool s8 = state != kAdam32;
        int i = 0;
        while (i < n) {
            int64_t items = 0;
            P.ndesc = 0;
            for (; i < n && P.ndesc < CAP; ++i) {
                const gq_adamw_tensor& T = t[i];
                if (T.numel == 0 || adam_state(T) != state) continue;
                AdamDesc& D = P.d[P.ndesc];
                D.p = T.p;
                D.g = T.g;
                D.m = T.m;
                D.v = T.v;
                D.ms = T.m_scale;
                D.vs = T.v_scale;
                D.copy = T.p_copy;
                D.numel = T.numel;
                D.wd = T.weight_decay;
                D.decay = (float)(1.0 - h->lr * T.weight_decay);
                D.key = (uint32_t)h->seed + (uint32_t)i * kAdamTensorMul;
                const size_t sa = s8 ? 8 : 16;
                const bool vec = aligned(T.p, 16) && aligned(T.g, 16) && aligned(T.m, sa) && aligned(T.v, sa) &&
                                 (!T.p_copy || aligned(T.p_copy, 16));
                D.flags = (T.p_dtype == GQ_BF16 ? kAdamPBf16 : 0) | (T.g_dtype == GQ_BF16 ? kAdamGBf16 : 0) |
                          (vec ? kAdamVec : 0);
                D.pad = 0;
                P.start[P.ndesc++] = items;
                items += (T.numel + kAdamItem - 1) / kAdamItem;
            }
            P.start[P.ndesc] = items;
            if (items == 0) continue;
            const unsigned blocks = (unsigned)std::min<int64_t>(items, (int64_t)sm_count() * 32);
            if (state == kAdam32) adamw_kernel<kAdam32, CAP><<<blocks, kAdamThreads, 0, stream>>>(P);
            else if (state == kAdam8Linear) adamw_kernel<kAdam8Linear, CAP><<<blocks, kAdamThreads, 0, stream>>>(P);
            else adamw_kernel<kAdam8Square, CAP><<<blocks, kAdamThreads, 0, stream>>>(P);
            if (launch_status() != GQ_OK) return GQ_ERR_CUDA;
        }
    }
    return GQ_OK;
}

}  // namespace

extern "C" gq_status gq_adamw_step(const gq_adamw_tensor* t, int n, const gq_adamw_hyper* h, cudaStream_t stream) {
    if (n < 0 || (n > 0 && !t) || !h) return GQ_ERR_INVALID_ARG;
    if (!(h->beta1 >= 0.0 && h->beta1 < 1.0) || !(h->beta2 >= 0.0 && h->beta2 < 1.0) || !(h->eps >= 0.0) ||
        !std::isfinite(h->eps) || !std::isfinite(h->lr) || (!h->d_step && h->step < 1))
        return GQ_ERR_INVALID_ARG;
    if ((h->d_step && !aligned(h->d_step, 8)) || (h->d_lr && !aligned(h->d_lr, 4)) ||
        (h->d_grad_scale && !aligned(h->d_grad_scale, 4)))
        return GQ_ERR_MISALIGNED;
    for (int i = 0; i < n; ++i) {
        const gq_status st = check_adamw(t[i]);
        if (st != GQ_OK) return st;
    }
    AdamStep S{};
    const int64_t step = h->d_step ? 1 : h->step;
    S.lr = h->lr;
    S.beta1 = h->beta1;
    S.beta2 = h->beta2;
    S.bias1 = 1.0 - std::pow(h->beta1, (double)step);
    S.b1 = (float)h->beta1;
    S.c1 = (float)(1.0 - h->beta1);
    S.b2 = (float)h->beta2;
    S.c2 = (float)(1.0 - h->beta2);
    S.eps = (float)h->eps;
    S.one = 1.0f;
    S.paired = S.eps <= kAdamHigh / 4.0f;
    S.inv_bc2 = (float)(1.0 / std::sqrt(1.0 - std::pow(h->beta2, (double)step)));
    S.step_size = (float)(h->lr / S.bias1);
    S.key_step = (uint32_t)step * kAdamStepMul;
    S.d_step = h->d_step;
    S.d_lr = h->d_lr;
    S.d_grad_scale = h->d_grad_scale;
    return n <= kAdamFew ? launch_adamw<kAdamFew>(t, n, h, S, stream) : launch_adamw<kAdamDesc>(t, n, h, S, stream);
}
