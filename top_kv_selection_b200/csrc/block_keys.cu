// block_keys.cu -- the indexer keys of whole blocks of tokens.
//
// A block's key is the mean of its m tokens' decoded indexer keys (FP8 codes
// times their scales; the Hadamard rotation is linear, so the mean of rotated
// keys is the rotated mean), quantised like a token's key by act_quant: scale
// max(amax, 1e-4) / 448, code e4m3_rn_satfinite(x / scale).  The entries are in
// the layout that the compressed-entry scorer and top-k take.
//
// A warp owns a block: one 16-byte load gives a lane 16 dims of a token, so
// D / 16 lanes cover a token and a warp 512 / D tokens per load.  Each lane
// sums its dims over its tokens in fp32, the token groups are added by
// shuffles in a fixed order.  Bound by the keys' bytes (D + 4 per token).
#include "common.cuh"
#include "quant.cuh"

namespace dsa {
namespace {

constexpr int kWarps = 8;

template <int D>
__global__ void __launch_bounds__(32 * kWarps)
block_keys_kernel(const uint8_t *__restrict__ k_cache, const float *__restrict__ k_scale, int64_t t_max,
                  int64_t first, int64_t per_seq, int64_t total, int block, uint8_t *__restrict__ blk_cache,
                  float *__restrict__ blk_scale, int64_t n_max) {
    constexpr int kLanes = D / 16, kTok = 32 / kLanes;
    const int lane = threadIdx.x & 31, piece = lane % kLanes, sub = lane / kLanes;
    const int64_t step = (int64_t)gridDim.x * kWarps;
    for (int64_t i = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5); i < total; i += step) {
        const int64_t b = i / per_seq, e = first + (i - b * per_seq);
        const int64_t t0 = b * t_max + e * block;
        float acc[16];
#pragma unroll
        for (int d = 0; d < 16; d++) acc[d] = 0.f;
#pragma unroll 4
        for (int j = sub; j < block; j += kTok) {
            const uint4 w = *reinterpret_cast<const uint4 *>(k_cache + (t0 + j) * D + 16 * piece);
            const float s = k_scale[t0 + j];
            const uint32_t ws[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
            for (int q = 0; q < 4; q++) {
                float f[4];
                e4m3x4_to_f32(ws[q], f[0], f[1], f[2], f[3]);
#pragma unroll
                for (int d = 0; d < 4; d++) acc[4 * q + d] = fmaf(f[d], s, acc[4 * q + d]);
            }
        }
        float amax = 0.f;
#pragma unroll
        for (int d = 0; d < 16; d++) {
#pragma unroll
            for (int m = kLanes; m < 32; m <<= 1) acc[d] += __shfl_xor_sync(0xffffffffu, acc[d], m);
            acc[d] = __fdiv_rn(acc[d], (float)block);
            amax = fmaxf(amax, fabsf(acc[d]));
        }
#pragma unroll
        for (int m = 1; m < kLanes; m <<= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, m));
        const float sc = __fdiv_rn(fmaxf(amax, 1e-4f), 448.0f), rs = __frcp_rn(sc);
        if (sub == 0) {
            uint32_t c[4];
#pragma unroll
            for (int q = 0; q < 4; q++)
                c[q] = e4m3x2_rn_sat(div_rn_by(acc[4 * q], sc, rs), div_rn_by(acc[4 * q + 1], sc, rs)) |
                       e4m3x2_rn_sat(div_rn_by(acc[4 * q + 2], sc, rs), div_rn_by(acc[4 * q + 3], sc, rs)) << 16;
            *reinterpret_cast<uint4 *>(blk_cache + (b * n_max + e) * D + 16 * piece) =
                make_uint4(c[0], c[1], c[2], c[3]);
            if (piece == 0) blk_scale[b * n_max + e] = sc;
        }
    }
}

}  // namespace
}  // namespace dsa

extern "C" dsa_status dsa_block_keys(const uint8_t *k_cache, const float *k_scale, int64_t t_max, int B,
                                     int64_t start_pos, int64_t S, int D, int block, uint8_t *blk_cache,
                                     float *blk_scale, int64_t n_max, dsa_stream_t stream) {
    if (B < 0 || S < 0 || start_pos < 0 || block < 1 || n_max < 0) return DSA_ERR_INVALID_ARG;
    if (D != 64 && D != 128) return DSA_ERR_UNSUPPORTED;
    if (start_pos + S > t_max) return DSA_ERR_INVALID_ARG;
    const int64_t first = start_pos / block, last = (start_pos + S) / block;
    if (last > n_max) return DSA_ERR_INVALID_ARG;
    if (B == 0 || last == first) return DSA_OK;
    if (!k_cache || !k_scale || !blk_cache || !blk_scale) return DSA_ERR_INVALID_ARG;
    if (!dsa::aligned16(k_cache) || !dsa::aligned16(blk_cache) || (reinterpret_cast<uintptr_t>(k_scale) & 3) ||
        (reinterpret_cast<uintptr_t>(blk_scale) & 3))
        return DSA_ERR_INVALID_ARG;
    const int64_t total = B * (last - first);
    const int64_t blocks = (total + dsa::kWarps - 1) / dsa::kWarps, cap = (int64_t)dsa::num_sms() * 8;
    const unsigned grid = (unsigned)(blocks < cap ? blocks : cap);
    const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    if (D == 128)
        dsa::block_keys_kernel<128><<<grid, 32 * dsa::kWarps, 0, st>>>(
            k_cache, k_scale, t_max, first, last - first, total, block, blk_cache, blk_scale, n_max);
    else
        dsa::block_keys_kernel<64><<<grid, 32 * dsa::kWarps, 0, st>>>(
            k_cache, k_scale, t_max, first, last - first, total, block, blk_cache, blk_scale, n_max);
    return dsa::launch_status();
}
