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
// sums its dims over its tokens in fp32, eight tokens' loads in flight; the
// token groups are added by shuffles in a fixed order.  Codes that the fp32
// mean leaves in doubt (about one block in 250) are taken from a mean in 64
// bits.  Bound by the keys' bytes (D + 4 per token).
#include "common.cuh"
#include "quant.cuh"

namespace dsa {
namespace {

constexpr int kWarps = 8;

// The mean of the block's keys in 64 bits, for the codes that fp32 leaves in
// doubt: dims [16 piece, 16 piece + 8 h + 8) of which this call sums the eight
// from 8 h on.
template <int D>
__device__ __noinline__ void exact_mean(const uint8_t *k_cache, const float *k_scale, int64_t t0, int block, int piece,
                                        int sub, int h, double (&acc)[8]) {
    constexpr int kLanes = D / 16, kTok = 32 / kLanes;
#pragma unroll
    for (int d = 0; d < 8; d++) acc[d] = 0.0;
    for (int j = sub; j < block; j += kTok) {
        const uint2 w = *reinterpret_cast<const uint2 *>(k_cache + (t0 + j) * D + 16 * piece + 8 * h);
        const double s = (double)k_scale[t0 + j];
        float f[8];
        e4m3x4_to_f32(w.x, f[0], f[1], f[2], f[3]);
        e4m3x4_to_f32(w.y, f[4], f[5], f[6], f[7]);
#pragma unroll
        for (int d = 0; d < 8; d++) acc[d] = fma((double)f[d], s, acc[d]);
    }
#pragma unroll
    for (int d = 0; d < 8; d++) {
#pragma unroll
        for (int m = kLanes; m < 32; m <<= 1) acc[d] += __shfl_xor_sync(0xffffffffu, acc[d], m);
        acc[d] /= block;
    }
}

template <int D>
__global__ void __launch_bounds__(32 * kWarps)
block_keys_kernel(const uint8_t *k_cache, const float *k_scale, int64_t t_max, int64_t first, int64_t per_seq,
                  int64_t total, int block, uint8_t *blk_cache, float *blk_scale, int64_t n_max) {
    constexpr int kLanes = D / 16, kTok = 32 / kLanes, kBatch = 8;
    const int lane = threadIdx.x & 31, piece = lane % kLanes, sub = lane / kLanes;
    const int64_t step = (int64_t)gridDim.x * kWarps;
    for (int64_t i = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5); i < total; i += step) {
        const int64_t b = i / per_seq, e = first + (i - b * per_seq);
        const int64_t t0 = b * t_max + e * block;
        const uint8_t *k0 = k_cache + t0 * D + 16 * piece;
        float acc[16];
#pragma unroll
        for (int d = 0; d < 16; d++) acc[d] = 0.f;
        for (int j0 = sub; j0 < block; j0 += kTok * kBatch) {
            uint4 w[kBatch];
            float s[kBatch];
#pragma unroll
            for (int u = 0; u < kBatch; u++) {
                const int j = j0 + u * kTok;
                w[u] = j < block ? *reinterpret_cast<const uint4 *>(k0 + (int64_t)j * D) : make_uint4(0, 0, 0, 0);
                s[u] = j < block ? k_scale[t0 + j] : 0.f;
            }
#pragma unroll
            for (int u = 0; u < kBatch; u++) {
                const uint32_t ws[4] = {w[u].x, w[u].y, w[u].z, w[u].w};
#pragma unroll
                for (int q = 0; q < 4; q++) {
                    float f[4];
                    e4m3x4_to_f32(ws[q], f[0], f[1], f[2], f[3]);
#pragma unroll
                    for (int d = 0; d < 4; d++) acc[4 * q + d] = fmaf(f[d], s[u], acc[4 * q + d]);
                }
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
        float sc = __fdiv_rn(fmaxf(amax, 1e-4f), 448.0f);
        const float rs = __frcp_rn(sc);
        // a quotient is in doubt when its fp32 error (2^-20 covers the sums of
        // blocks of any usual length) reaches over a border between two codes
        uint32_t c[4];
        bool doubt = false;
#pragma unroll
        for (int q = 0; q < 4; q++) {
            uint32_t lo = 0, hi = 0;
#pragma unroll
            for (int d = 0; d < 4; d += 2) {
                const float q0 = acc[4 * q + d] * rs, q1 = acc[4 * q + d + 1] * rs;
                lo |= e4m3x2_rn_sat(fmaf(q0, -0x1p-20f, q0), fmaf(q1, -0x1p-20f, q1)) << (8 * d);
                hi |= e4m3x2_rn_sat(fmaf(q0, 0x1p-20f, q0), fmaf(q1, 0x1p-20f, q1)) << (8 * d);
            }
            doubt |= lo != hi;
            c[q] = lo;
        }
        if (__any_sync(0xffffffffu, doubt)) {
            double m0[8], m1[8], top = 0.0;
            exact_mean<D>(k_cache, k_scale, t0, block, piece, sub, 0, m0);
            exact_mean<D>(k_cache, k_scale, t0, block, piece, sub, 1, m1);
#pragma unroll
            for (int d = 0; d < 8; d++) top = fmax(top, fmax(fabs(m0[d]), fabs(m1[d])));
#pragma unroll
            for (int m = 1; m < kLanes; m <<= 1) top = fmax(top, __shfl_xor_sync(0xffffffffu, top, m));
            sc = __double2float_rn(fmax(top, (double)1e-4f) / 448.0);
#pragma unroll
            for (int q = 0; q < 4; q++) {
                float f[4];
#pragma unroll
                for (int d = 0; d < 4; d++) f[d] = __double2float_rn((q < 2 ? m0[4 * q + d] : m1[4 * (q & 1) + d]) / sc);
                c[q] = e4m3x2_rn_sat(f[0], f[1]) | e4m3x2_rn_sat(f[2], f[3]) << 16;
            }
        }
        if (sub == 0) {
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
    const int64_t blocks = (total + dsa::kWarps - 1) / dsa::kWarps, cap = 1 << 20;
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
