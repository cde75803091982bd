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
// sums its dims over its tokens in fp32 (packed pairs, up to sixteen tokens'
// loads in flight: 138 MB of keys take 29.7 us; eight at a time cost 3 more); the lanes of a token group then trade halves until each holds the
// sums of D / 32 dims, in a fixed order.  Codes that the fp32 mean leaves in
// doubt are taken from a mean in 64 bits (about one block in 30).  The keys'
// bytes (D + 4 per token) bound it from below; the decoding of the codes, some
// ten instructions a token and warp, comes close.
#include <type_traits>

#include "common.cuh"
#include "quant.cuh"

namespace dsa {
namespace {

constexpr int kWarps = 8;

template <int D>
__global__ void __launch_bounds__(32 * kWarps, 3)
block_keys_kernel(const uint8_t *__restrict__ k_cache, const float *__restrict__ k_scale, int64_t t_max, int64_t first,
                  int64_t per_seq, int64_t total, int block, uint8_t *__restrict__ blk_cache,
                  float *__restrict__ blk_scale, int64_t n_max) {
    constexpr int kLanes = D / 16, kTok = 32 / kLanes, kOwn = D / 32;
    const int lane = threadIdx.x & 31, piece = lane % kLanes, sub = lane / kLanes;
    const int64_t i = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5);
    if (i >= total) return;
    const int64_t b = i / per_seq, e = first + (i - b * per_seq);
    const int64_t t0 = b * t_max + e * block;
    const uint8_t *kp = k_cache + (t0 + sub) * D + 16 * piece;
    const float *sp = k_scale + t0 + sub;
    float2 acc[8];
#pragma unroll
    for (int d = 0; d < 8; d++) acc[d] = make_float2(0.f, 0.f);
    auto add = [&](const uint4 &w, float s) {
        const uint32_t ws[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int q = 0; q < 4; q++) {
            float f[4];
            e4m3x4_to_f32(ws[q], f[0], f[1], f[2], f[3]);
            acc[2 * q] = __ffma2_rn(make_float2(f[0], f[1]), make_float2(s, s), acc[2 * q]);
            acc[2 * q + 1] = __ffma2_rn(make_float2(f[2], f[3]), make_float2(s, s), acc[2 * q + 1]);
        }
    };
    // n tokens of this lane, their loads in flight together
    int j = sub;
    auto batch = [&](auto n) {
        constexpr int kN = decltype(n)::value;
        for (; j + (kN - 1) * kTok < block; j += kTok * kN, kp += kTok * kN * D, sp += kTok * kN) {
            uint4 w[kN];
            float s[kN];
#pragma unroll
            for (int u = 0; u < kN; u++) {
                w[u] = *reinterpret_cast<const uint4 *>(kp + u * kTok * D);
                s[u] = sp[u * kTok];
            }
#pragma unroll
            for (int u = 0; u < kN; u++) add(w[u], s[u]);
        }
    };
    batch(std::integral_constant<int, 16>());
    batch(std::integral_constant<int, 4>());
    batch(std::integral_constant<int, 1>());
    __syncwarp();
    // trade halves: the lane whose bit is set keeps the upper half of its dims
    float v[16];
#pragma unroll
    for (int d = 0; d < 8; d++) {
        v[2 * d] = acc[d].x;
        v[2 * d + 1] = acc[d].y;
    }
#pragma unroll
    for (int m = 16, n = 8; m >= kLanes; m >>= 1, n >>= 1) {
        const bool up = lane & m;
#pragma unroll
        for (int d = 0; d < n; d++) {
            const float give = up ? v[d] : v[d + n], keep = up ? v[d + n] : v[d];
            v[d] = keep + __shfl_xor_sync(0xffffffffu, give, m);
        }
    }
    // this lane's dims (bits 4, 3 and for D = 64 bit 2 of the lane, from the top)
    int own = 16 * piece;
#pragma unroll
    for (int m = 16, n = 8; m >= kLanes; m >>= 1, n >>= 1) own += lane & m ? n : 0;
    const float inv = 1.f / (float)block;
    float amax = 0.f;
#pragma unroll
    for (int d = 0; d < kOwn; d++) {
        v[d] *= inv;
        amax = fmaxf(amax, fabsf(v[d]));
    }
    amax = warp_max(amax);
    float sc = __fdiv_rn(fmaxf(amax, 1e-4f), 448.0f);
    const float rs = __frcp_rn(sc);
    // A quotient is in doubt when its fp32 error may reach over a border between
    // two codes: 2^-21 of the vector's largest (448), since the sum's error goes
    // by its terms and not by what they cancel to, and 2^-20 of itself.
    constexpr float kAbs = 448.f * 0x1p-21f;
    uint32_t lo = 0, hi = 0;
#pragma unroll
    for (int d = 0; d < kOwn; d += 2) {
        const float q0 = v[d] * rs, q1 = v[d + 1] * rs;
        const float d0 = fmaf(fabsf(q0), 0x1p-20f, kAbs), d1 = fmaf(fabsf(q1), 0x1p-20f, kAbs);
        lo |= e4m3x2_rn_sat(q0 - d0, q1 - d1) << (8 * d);
        hi |= e4m3x2_rn_sat(q0 + d0, q1 + d1) << (8 * d);
    }
    if (__any_sync(0xffffffffu, lo != hi)) {
        double x[kOwn], top = 0.0;
#pragma unroll
        for (int d = 0; d < kOwn; d++) x[d] = 0.0;
        const uint8_t *k0 = k_cache + t0 * D + own;
#pragma unroll 16
        for (int t = 0; t < block; t++) {
            const double s = (double)k_scale[t0 + t];
            uint32_t w;
            if constexpr (kOwn == 4)
                w = *reinterpret_cast<const uint32_t *>(k0 + (int64_t)t * D);
            else
                w = *reinterpret_cast<const uint16_t *>(k0 + (int64_t)t * D);
            float f[4];
            e4m3x4_to_f32(w, f[0], f[1], f[2], f[3]);
#pragma unroll
            for (int d = 0; d < kOwn; d++) x[d] = fma((double)f[d], s, x[d]);
        }
#pragma unroll
        for (int d = 0; d < kOwn; d++) {
            x[d] /= block;
            top = fmax(top, fabs(x[d]));
        }
#pragma unroll
        for (int m = 1; m < 32; m <<= 1) top = fmax(top, __shfl_xor_sync(0xffffffffu, top, m));
        const double exact = fmax(top, (double)1e-4f) / 448.0;
        sc = __double2float_rn(exact);
        lo = 0;
#pragma unroll
        for (int d = 0; d < kOwn; d += 2)
            lo |= e4m3x2_rn_sat(__double2float_rn(x[d] / exact), __double2float_rn(x[d + 1] / exact)) << (8 * d);
    }
    uint8_t *dst = blk_cache + (b * n_max + e) * D + own;
    if constexpr (kOwn == 4)
        *reinterpret_cast<uint32_t *>(dst) = lo;
    else
        *reinterpret_cast<uint16_t *>(dst) = (uint16_t)lo;
    if (lane == 0) blk_scale[b * n_max + e] = sc;
}

}  // namespace
}  // namespace dsa

extern "C" dsa_status dsa_block_keys(const uint8_t *k_cache, const float *k_scale, int64_t t_max, int B,
                                     int64_t start_pos, int64_t S, int D, int block, uint8_t *blk_cache,
                                     float *blk_scale, int64_t n_max, dsa_stream_t stream) {
    if (B < 0 || S < 0 || start_pos < 0 || block < 1 || n_max < 0 || t_max < 0) return DSA_ERR_INVALID_ARG;
    if (D != 64 && D != 128) return DSA_ERR_UNSUPPORTED;
    if (start_pos > t_max - S) return DSA_ERR_INVALID_ARG;
    const int64_t first = start_pos / block, last = (start_pos + S) / block;
    if (last > n_max) return DSA_ERR_INVALID_ARG;
    if (B == 0 || last == first) return DSA_OK;
    if (!k_cache || !k_scale || !blk_cache || !blk_scale) return DSA_ERR_INVALID_ARG;
    if (!dsa::aligned16(k_cache) || !dsa::aligned16(blk_cache) || (reinterpret_cast<uintptr_t>(k_scale) & 3) ||
        (reinterpret_cast<uintptr_t>(blk_scale) & 3))
        return DSA_ERR_INVALID_ARG;
    if (last - first > (int64_t)INT32_MAX * dsa::kWarps / B) return DSA_ERR_UNSUPPORTED;     // more than a grid
    const int64_t total = B * (last - first);
    const int64_t blocks = (total + dsa::kWarps - 1) / dsa::kWarps;
    const unsigned grid = (unsigned)blocks;
    const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    if (D == 128)
        dsa::block_keys_kernel<128><<<grid, 32 * dsa::kWarps, 0, st>>>(
            k_cache, k_scale, t_max, first, last - first, total, block, blk_cache, blk_scale, n_max);
    else
        dsa::block_keys_kernel<64><<<grid, 32 * dsa::kWarps, 0, st>>>(
            k_cache, k_scale, t_max, first, last - first, total, block, blk_cache, blk_scale, n_max);
    return dsa::launch_status();
}
