// gq_linear.cu -- host side of gq_tile_weight, gq_gemm_epilogue and
// gq_gemm_grouped (include/gq.h): argument checks, launch planning, launches.
#include <algorithm>
#include <atomic>
#include <cstring>

#include "gq_host.h"
#include "gq_linear.cuh"

namespace {

using namespace gq;

constexpr int kLinSmem = 112 * 1024;     // a block's share of an SM that holds two

static_assert(sizeof(gq_epilogue) == 40, "the layout is part of the ABI (the Python binding mirrors it)");

// Launch of linear_kernel with clusters of `cluster` blocks, as a kernel whose blocks may start before the one ahead of
// it in the stream has ended (one token through 1536 x 512: a tenth less time a call in a row of calls).
gq_status launch_next(void (*kernel)(LinParams), const LinParams& P, int64_t blocks, int threads, int smem, int cluster,
                      cudaStream_t stream) {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)blocks);
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = (size_t)smem;
    cfg.stream = stream;
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    at[1].id = cudaLaunchAttributeClusterDimension;
    at[1].val.clusterDim = {(unsigned)cluster, 1, 1};
    cfg.attrs = at;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    return cuda_status(cudaLaunchKernelEx(&cfg, kernel, P));
}

// X [M, K] as a tensor map with a box of 64 columns x `rows` rows; zeros past the ends.
bool map_x(CUtensorMap* map, const void* d_x, int64_t M, int64_t K, int64_t ldx, int rows) {
    PFN_cuTensorMapEncodeTiled enc = encode_tiled();
    if (!enc) return false;
    const cuuint64_t dim[2] = {(cuuint64_t)K, (cuuint64_t)M};
    const cuuint64_t stride[1] = {(cuuint64_t)ldx * 2};
    const cuuint32_t box[2] = {(cuuint32_t)kLinK, (cuuint32_t)rows};
    const cuuint32_t step[2] = {1, 1};
    return enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(d_x), dim, stride, box, step,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int QB, int NT>
gq_status launch(LinParams& P, const void* d_x, int64_t K, int64_t ldx, cudaStream_t stream) {
    using S = LinShape<QB, NT>;
    static std::atomic<bool> set[kMaxDevices];
    if (!map_x(&P.tmap_x, d_x, P.M, K, ldx, NT)) return GQ_ERR_UNSUPPORTED;
    P.idesc = gemm_idesc(kLinRows, NT);
    // token tiles: exact for one weight; for experts the most that any offsets can give
    const int64_t tts = P.offsets ? P.M / NT + std::min<int64_t>(P.E, P.M) : (P.M + NT - 1) / NT;
    const int64_t units = tts * P.rts;
    if (units > INT32_MAX) return GQ_ERR_UNSUPPORTED;
    // The split: blocks for every SM once, as far as a cluster of 4 (of 8 where a tile or few are all there is: clusters
    // of 8 find room on fewer SMs); then twice, if each block keeps 12 column blocks to stream.  N = K = 2048, M 16:
    // 11.1, 8.5, 7.0, 7.8 us with 1, 2, 4, 8 blocks a tile; N = K = 8192: 32.7, 20.7, 18.1, 23.9; N 1792, K 512, M 333:
    // 9.2, 8.8, 10.4, 19.4.
    const int64_t sms = sm_count();
    int ls = 0;
    while (ls < (units <= 8 ? 3 : 2) && (units << (ls + 1)) <= sms && P.kbs >= 2 << (ls + 1)) ++ls;
    if (ls < 2 && (units << (ls + 1)) <= 2 * sms && P.kbs >= 12 << (ls + 1)) ++ls;
    if (units << ls > INT32_MAX) return GQ_ERR_UNSUPPORTED;
    P.log_split = ls;
    const int split = 1 << ls;
    // two blocks to an SM
    P.stages = std::min<int>(kLinMaxStages, (kLinSmem - S::smem(0)) / (int)S::stage);
    if (P.stages < (int)S::slots) return GQ_ERR_UNSUPPORTED;   // never: the conversion's waits need it
    const int smem = std::max(S::smem(P.stages), split > 1 ? S::smem(0) + NT * kLinRows * 4 : 0);
    int dev = 0;
    if (cuda_status(cudaGetDevice(&dev)) != GQ_OK) return GQ_ERR_CUDA;
    if (dev >= kMaxDevices || !set[dev].load(std::memory_order_relaxed)) {
        if (cuda_status(cudaFuncSetAttribute(linear_kernel<QB, NT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             kLinSmem)) != GQ_OK)
            return GQ_ERR_CUDA;
        if (dev < kMaxDevices) set[dev].store(true, std::memory_order_relaxed);
    }
    return launch_next(linear_kernel<QB, NT>, P, units * split, S::threads, smem, split, stream);
}

// Whether the pair kernel is the faster one.  Three conditions, measured in us, pairs against one block a tile:
//  - Units that fill the pairs' rounds to three fifths: N = K = 8192: M 256 (fill 0.43) 45.3 / 37.6, M 320 (0.86) 37.6 / 63.3.
//  - 24 column blocks in all for a pair, so that its first unit's way through the pipeline counts for little: N 4096, K
//    1024: M 1024 (16) 14.1 / 13.6, M 2048 (32) 19.9 / 24.4; N 24576, K 256, M 256 (8) 14.3 / 11.6; 16 experts of 1584 x
//    528, 256 rows each (18) 20.8 / 18.9; N 4096, K 200, M 8192 (28) 35.9 / 45.2.
//  - Enough rows that a converted code serves more tokens than in the other kernel's tiles of up to 128, or nearly: N
//    32768, K 1024: M 128 16.0 / 13.5, M 192 17.7 / 23.2; with long K from 96 rows on, N 16384, K 8192: M 64 35.8 / 29.3, M
//    96 37.0 / 39.4, K 2048: M 128 14.9 / 16.3 (N 32768, K 1536: 19.8 / 17.4); experts, whose counts differ, from 96 rows on average, 2048 x 1024: 64 rows 18.3 / 16.9, 96 rows
//    17.6 / 21.1, and from 64 where there is much of it, 64 experts of 4096 x 2048: 48 rows 145.8 / 142.1, 64 rows
//    141.1 / 165.5.
bool pair_pays(const LinParams& P) {
    const int64_t rows = (P.M + P.E - 1) / P.E, pairs = std::max(1, sm_count() / 2);
    const int64_t units = (P.rts + 1) / 2 * (int64_t)P.E * ((rows + kPairNT - 1) / kPairNT);
    const int64_t rounds = (units + pairs - 1) / pairs;
    const int least = P.E == 1 ? (P.kbs < 32 ? 129 : 96) : (rounds >= 4 && P.kbs >= 16 ? 64 : 96);
    return rows >= least && 5 * units >= 3 * rounds * pairs && rounds * P.kbs >= 24;
}

// The kernel of 256 x 256 tiles over pairs of SMs.
template <int QB>
gq_status launch_pair(LinParams& P, const void* d_x, int64_t K, int64_t ldx, cudaStream_t stream) {
    using S = PairShape<QB>;
    static std::atomic<bool> set[kMaxDevices];
    if (!map_x(&P.tmap_x, d_x, P.M, K, ldx, kPairNT / 2)) return GQ_ERR_UNSUPPORTED;
    constexpr int smem = S::smem(S::stages);
    int dev = 0;
    if (cuda_status(cudaGetDevice(&dev)) != GQ_OK) return GQ_ERR_CUDA;
    if (dev >= kMaxDevices || !set[dev].load(std::memory_order_relaxed)) {
        if (cuda_status(cudaFuncSetAttribute(linear_pair_kernel<QB>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             smem)) != GQ_OK)
            return GQ_ERR_CUDA;
        if (dev < kMaxDevices) set[dev].store(true, std::memory_order_relaxed);
    }
    // as many pairs as have work (for experts, at most); 32-bit unit numbers
    const int64_t tts = P.offsets ? P.M / kPairNT + std::min<int64_t>(P.E, P.M) : (P.M + kPairNT - 1) / kPairNT;
    const int64_t units = tts * ((P.rts + 1) / 2);
    if (units > INT32_MAX / 2) return GQ_ERR_UNSUPPORTED;
    const int64_t pairs = std::min<int64_t>(units, sm_count() / 2);
    if ((units / pairs + 1) * ((P.kbs + 1) / 2) > INT32_MAX / 2) return GQ_ERR_UNSUPPORTED;   // stages are counted in 32 bits
    linear_pair_kernel<QB><<<(unsigned)(2 * pairs), kPairThreads, smem, stream>>>(P);
    return launch_status();
}

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
    // a residual that is Y itself is read and written by the same thread, which wants the same elements
    if (e.residual && e.residual == d_y && (e.residual_dtype != e.y_dtype || (M > 1 && e.ldr != ldy)))
        return GQ_ERR_INVALID_ARG;
    if (d_status && !aligned(d_status, 4)) return GQ_ERR_MISALIGNED;
    const bool empty = M == 0 || N == 0 || E == 0;
    if (!empty) {
        if (!d_y || !d_scale_f16 || (K > 0 && (!d_x || !d_tiles))) return GQ_ERR_INVALID_ARG;
        auto size = [](int32_t d) { return d == GQ_F32 ? 4 : 2; };
        if ((K > 0 && (!aligned(d_x, 16) || (ldx % 8) != 0 || !aligned(d_tiles, 16))) || !aligned(d_scale_f16, 2) ||
            !aligned(d_y, size(e.y_dtype)) || (e.bias && !aligned(e.bias, size(e.bias_dtype))) ||
            (e.residual && !aligned(e.residual, size(e.residual_dtype))))
            return GQ_ERR_MISALIGNED;
    }
    if (!aligned(d_offsets, 4)) return GQ_ERR_MISALIGNED;
    if (d_status && cuda_status(cudaMemsetAsync(d_status, 0, sizeof(int32_t), stream)) != GQ_OK) return GQ_ERR_CUDA;
    LinParams P;
    std::memset(&P, 0, sizeof(P));
    if (empty) {
        // nothing to compute, but offsets that leave the batch are reported here too
        if (!d_offsets || !d_status || E == 0) return GQ_OK;
        P.offsets = d_offsets;
        P.status = d_status;
        P.M = M;
        P.E = E;
        linear_empty_kernel<<<1, 256, 0, stream>>>(P);     // (P.N is 0: no row is looked at)
        return launch_status();
    }
    P.tiles = d_tiles;
    P.scale = d_scale_f16;
    P.offsets = d_offsets;
    P.status = d_status;
    P.M = M;
    P.N = N;
    P.E = E;
    P.kbs = (int32_t)((K + kLinK - 1) / kLinK);
    P.rts = (int32_t)((N + kLinRows - 1) / kLinRows);
    P.epi = LinEpi{e.bias, e.residual, d_y, e.ldr, ldy, e.bias_dtype == GQ_BF16, e.residual_dtype == GQ_BF16,
                   e.y_dtype == GQ_BF16, e.act};
    if (K == 0) {
        linear_empty_kernel<<<(unsigned)std::min<int64_t>(M, 65535), 256, 0, stream>>>(P);
        return launch_status();
    }
    if (pair_pays(P)) return qbits == 6 ? launch_pair<6>(P, d_x, K, ldx, stream) : launch_pair<8>(P, d_x, K, ldx, stream);
    // tokens of a tile: the rows an expert has on average, rounded up to 16 .. 128
    const int64_t rows = (M + E - 1) / E;
    const int nt = rows <= 16 ? 16 : rows <= 32 ? 32 : rows <= 64 ? 64 : 128;
    if (qbits == 6)
        return nt == 16 ? launch<6, 16>(P, d_x, K, ldx, stream) : nt == 32 ? launch<6, 32>(P, d_x, K, ldx, stream)
             : nt == 64 ? launch<6, 64>(P, d_x, K, ldx, stream) : launch<6, 128>(P, d_x, K, ldx, stream);
    return nt == 16 ? launch<8, 16>(P, d_x, K, ldx, stream) : nt == 32 ? launch<8, 32>(P, d_x, K, ldx, stream)
         : nt == 64 ? launch<8, 64>(P, d_x, K, ldx, stream) : launch<8, 128>(P, d_x, K, ldx, stream);
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
