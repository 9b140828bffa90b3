// gq_linear.cu -- host side of gq_tile_weight, gq_gemm_epilogue and
// gq_gemm_grouped (include/gq.h): argument checks, launch planning, launches.
#include <algorithm>
#include <cstring>

#include "gq_host.h"
#include "gq_linear.cuh"

namespace {

using namespace gq;

static_assert(sizeof(gq_epilogue) == 40, "the layout is part of the ABI (the Python binding mirrors it)");

gq_status linear(const void* d_x, int64_t M, int64_t K, int64_t ldx, const int32_t* d_offsets, int64_t E,
                 const uint8_t* d_tiles, const uint16_t* d_scale_f16, int qbits, int64_t N, const gq_epilogue* epi,
                 void* d_y, int64_t ldy, int32_t* d_status, cudaStream_t stream) {
    const gq_epilogue none{nullptr, nullptr, 0, GQ_F32, GQ_F32, GQ_ACT_NONE, GQ_F32};
    const gq_epilogue& e = epi ? *epi : none;
    if (M < 0 || N < 0 || K < 0 || (qbits != 6 && qbits != 8)) return GQ_ERR_INVALID_ARG;
    if (ldx < K || ldy < N || (e.residual && e.ldr < N)) return GQ_ERR_INVALID_ARG;
    if (e.act < GQ_ACT_NONE || e.act > GQ_ACT_GELU_TANH) return GQ_ERR_INVALID_ARG;
    auto known = [](int32_t d) { return d == GQ_F32 || d == GQ_BF16; };
    if (!known(e.y_dtype) || (e.bias && !known(e.bias_dtype)) || (e.residual && !known(e.residual_dtype)))
        return GQ_ERR_INVALID_ARG;
    if (M > INT32_MAX || K > INT32_MAX - 64 || N > INT32_MAX - 128 || E > 65535) return GQ_ERR_UNSUPPORTED;
    if (ldx > INT64_MAX / 16 / (M + 1) || ldy > INT64_MAX / 16 / (M + 1) ||
        (e.residual && e.ldr > INT64_MAX / 16 / (M + 1)))
        return GQ_ERR_INVALID_ARG;
    if (d_status && !aligned(d_status, 4)) return GQ_ERR_MISALIGNED;
    const bool empty = M == 0 || N == 0 || E == 0;
    if (!empty) {
        if (!d_y || !d_scale_f16 || (K > 0 && (!d_x || !d_tiles))) return GQ_ERR_INVALID_ARG;
        auto size = [](int32_t d) { return d == GQ_F32 ? 4 : 2; };
        if ((K > 0 && (!aligned(d_x, 16) || (ldx % 8) != 0 || !aligned(d_tiles, 16))) || !aligned(d_scale_f16, 2) ||
            !aligned(d_y, size(e.y_dtype)) || (e.bias && !aligned(e.bias, size(e.bias_dtype))) ||
            (e.residual && !aligned(e.residual, size(e.residual_dtype))) || !aligned(d_offsets, 4))
            return GQ_ERR_MISALIGNED;
    }
    if (d_status && cuda_status(cudaMemsetAsync(d_status, 0, sizeof(int32_t), stream)) != GQ_OK) return GQ_ERR_CUDA;
    if (empty) return GQ_OK;
    LinParams P;
    std::memset(&P, 0, sizeof(P));
    P.x = static_cast<const uint16_t*>(d_x);
    P.tiles = d_tiles;
    P.scale = d_scale_f16;
    P.offsets = d_offsets;
    P.status = d_status;
    P.M = M;
    P.N = N;
    P.K = K;
    P.ldx = ldx;
    P.kbs = (K + kLinK - 1) / kLinK;
    P.rts = (N + kLinRows - 1) / kLinRows;
    P.E = E;
    P.epi = LinEpi{e.bias, e.residual, d_y, e.ldr, ldy, e.bias_dtype == GQ_BF16, e.residual_dtype == GQ_BF16,
                   e.y_dtype == GQ_BF16, e.act};
    const dim3 grid((unsigned)P.rts, (unsigned)std::min<int64_t>((M + 7) / 8, 64), (unsigned)E);
    if (qbits == 6) linear_kernel<6><<<grid, kLinRows, 0, stream>>>(P);
    else linear_kernel<8><<<grid, kLinRows, 0, stream>>>(P);
    return launch_status();
}

}  // namespace

extern "C" {

int64_t gq_tile_bytes(int64_t N, int64_t K, int qbits) {
    if (N < 0 || K < 0 || N > INT32_MAX - 128 || K > INT32_MAX - 64 || (qbits != 6 && qbits != 8)) return -1;
    return (N + kLinRows - 1) / kLinRows * ((K + kLinK - 1) / kLinK) * lin_block_bytes(qbits);
}

gq_status gq_tile_weight(const uint8_t* d_packed, int64_t E, int64_t N, int64_t K, int qbits, uint8_t* d_tiles,
                         cudaStream_t stream) {
    if (E < 0 || N < 0 || K < 0 || (qbits != 6 && qbits != 8)) return GQ_ERR_INVALID_ARG;
    if (gq_tile_bytes(N, K, qbits) < 0 || E > 65535) return GQ_ERR_UNSUPPORTED;
    if (E == 0 || N == 0 || K == 0) return GQ_OK;
    if (!d_packed || !d_tiles) return GQ_ERR_INVALID_ARG;
    if (!aligned(d_tiles, 16)) return GQ_ERR_MISALIGNED;
    const int64_t kbs = (K + kLinK - 1) / kLinK, blocks = E * ((N + kLinRows - 1) / kLinRows) * kbs;
    if (blocks > INT32_MAX) return GQ_ERR_UNSUPPORTED;
    tile_weight_kernel<<<(unsigned)blocks, kLinRows, 0, stream>>>(d_packed, N, K, packed_row_bytes(K, qbits), qbits,
                                                                  kbs, d_tiles);
    return launch_status();
}

gq_status gq_gemm_epilogue(const void* d_x, int64_t M, int64_t K, int64_t ldx, const uint8_t* d_tiles,
                           const uint16_t* d_scale_f16, int qbits, int64_t N, const gq_epilogue* epi, void* d_y,
                           int64_t ldy, int32_t* d_status, cudaStream_t stream) {
    return linear(d_x, M, K, ldx, nullptr, 1, d_tiles, d_scale_f16, qbits, N, epi, d_y, ldy, d_status, stream);
}

gq_status gq_gemm_grouped(const void* d_x, int64_t M, int64_t K, int64_t ldx, const int32_t* d_offsets, int64_t E,
                          const uint8_t* d_tiles, const uint16_t* d_scale_f16, int qbits, int64_t N,
                          const gq_epilogue* epi, void* d_y, int64_t ldy, int32_t* d_status, cudaStream_t stream) {
    if (E < 0 || (E > 0 && M > 0 && N > 0 && !d_offsets)) return GQ_ERR_INVALID_ARG;
    return linear(d_x, M, K, ldx, d_offsets, E, d_tiles, d_scale_f16, qbits, N, epi, d_y, ldy, d_status, stream);
}

}  // extern "C"
