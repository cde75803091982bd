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
// loads in flight, chains of sixteen and a chain of their sums, which is kept in
// shared memory); the lanes of a token group then trade halves until each
// holds the sums of D / 32 dims, in a fixed order.
//
// An fp32 sum's error goes by its terms and not by what is left of them when
// tokens cancel, so the warp carries a bound on the terms, from the scales
// alone, and takes dims whose code that leaves in doubt again in 64 bits: at 64
// random tokens a block, about one dim in every third block.  Where the bound
// passes 2^-14 of the largest dim, the scale's dim is among them.  138 MB of
// keys in blocks of 64 tokens take 30.2 us, in blocks of 128 or 256 28.6, of 16
// 43.6, of 2048 127 (64 blocks a sequence leave most SMs idle; with one chain a
// lane, whose bound puts every dim in doubt there, 230); sums in 64 bits
// throughout (two more integer instructions a code) took 38 us at 64 and 105 at
// 2048.  The keys' bytes (D + 4 per token) bound it from
// below; the decoding of the codes, some ten instructions a token and warp,
// comes close.
#include <type_traits>

#include "common.cuh"
#include "quant.cuh"

namespace dsa {
namespace {

// A warp that takes dims again holds its block's place: two warps a block 30.2, eight
// 34.1 us (138 MB, 64 tokens a block).
constexpr int kWarps = 2;
constexpr int kFew = 16;         // dims that are worth a round of eight lanes each

// x as fp32 for the rounding to a code: cut, with a bit that says so, so that the
// code is that of x (not of x rounded to fp32 first).
__device__ __forceinline__ float f32_odd(double x) {
    const float f = __double2float_rz(x);
    return (double)f == x ? f : __uint_as_float(__float_as_uint(f) | 1u);
}

template <int D>
__global__ void __launch_bounds__(32 * kWarps, 16)
block_keys_kernel(const uint8_t *__restrict__ k_cache, const float *__restrict__ k_scale, int64_t t_max, int64_t first,
                  int64_t per_seq, int64_t total, int block, uint8_t *__restrict__ blk_cache,
                  float *__restrict__ blk_scale, int64_t n_max) {
    constexpr int kLanes = D / 16, kTok = 32 / kLanes, kOwn = D / 32;
    __shared__ float2 total_sm[kWarps][8][32];
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
    // of the scales: the sum of the chains before, this chain's, and the sum of all
    // partial sums (the error's bound)
    float sum_s = 0.f, sum_b = 0.f, sum_p = 0.f;
    auto add = [&](const uint4 &w, float s) {
        const uint32_t ws[4] = {w.x, w.y, w.z, w.w};
        sum_b += fabsf(s);
        sum_p += sum_b;
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
            if (kN == 16 && j + kTok * kN < block) {
                // chains of sixteen, and a sum of them, in shared memory
                sum_s += sum_b;
                sum_p += sum_s;
                sum_b = 0.f;
#pragma unroll
                for (int d = 0; d < 8; d++) {
                    float2 &t = total_sm[threadIdx.x >> 5][d][lane];
                    t = j == sub ? acc[d] : make_float2(t.x + acc[d].x, t.y + acc[d].y);
                    acc[d] = make_float2(0.f, 0.f);
                }
            }
        }
    };
    batch(std::integral_constant<int, 16>());
    batch(std::integral_constant<int, 4>());
    batch(std::integral_constant<int, 1>());
    if (sub + 16 * kTok < block) {
        sum_p += sum_s + sum_b;
#pragma unroll
        for (int d = 0; d < 8; d++) {
            const float2 t = total_sm[threadIdx.x >> 5][d][lane];
            acc[d] = make_float2(t.x + acc[d].x, t.y + acc[d].y);
        }
    }
    sum_s += sum_b;
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
    // How far the fp32 means may be off.  A term is at most 448 of its scale, so a
    // chain's partial sums are at most 448 of its scales' partial sums, and each step
    // is off by 2^-24 of one, the sum of the chains' too; a trade by 2^-24 of the sum so far, as are the two
    // roundings of the mean.  (A sixteenth more for the roundings of the bound.)
    constexpr int kTrades = kTok == 8 ? 3 : 2;
    float err = sum_p + (kTrades + 2) * sum_s;
#pragma unroll
    for (int m = 16; m >= kLanes; m >>= 1) err += __shfl_xor_sync(0xffffffffu, err, m);
    err *= inv * (448.f * 0x1.1p-24f);
    float sc = __fdiv_rn(fmaxf(amax, 1e-4f), 448.0f);
    const float rs = __frcp_rn(sc);
    // A code is in doubt where that error, of the mean and of the scale, may reach
    // over a border (a zero's sign does not count); a dim may be the largest where it
    // reaches the largest, which the scale's floor may make idle.  (Comparisons are
    // such that NaN, and a sum that leaves fp32's range, put a dim in doubt.)
    float far = err * rs;
    far = fmaf(far, far * (2.f / 448.f), far);
    const float rel = fmaf(far, 1.f / 448.f, 0x1p-21f);
    const bool floor = amax + 2.f * err < 1e-4f;
    uint32_t codes = 0, todo = 0;
#pragma unroll
    for (int d = 0; d < kOwn; d += 2) {
        const float q0 = v[d] * rs, q1 = v[d + 1] * rs;
        const float d0 = fmaf(fabsf(q0), rel, far), d1 = fmaf(fabsf(q1), rel, far);
        const uint32_t lo = e4m3x2_rn_sat(q0 - d0, q1 - d1), hi = e4m3x2_rn_sat(q0 + d0, q1 + d1);
        const uint32_t off = lo ^ hi, mag = (lo | hi) & 0x7F7F;
        codes |= e4m3x2_rn_sat(q0, q1) << (8 * d);
        todo |= (uint32_t)((off & 0xFF) && (mag & 0xFF)) << d;
        todo |= (uint32_t)((off >> 8) && (mag >> 8)) << (d + 1);
    }
    if (__any_sync(0xffffffffu, todo != 0 || !(floor || (err < amax * 0x1p-14f && amax < INFINITY)))) {
        // Those dims in 64 bits, and the largest one for the scale.
        const float least = amax == INFINITY ? 0.f : floor ? INFINITY : amax - 2.125f * err;
        uint32_t left[kOwn];
        int n = 0;
        double x[kOwn], top = 0.0;
#pragma unroll
        for (int d = 0; d < kOwn; d++) {
            todo |= (uint32_t)!(fabsf(v[d]) < least) << d;
            left[d] = __ballot_sync(0xffffffffu, todo >> d & 1);
            n += __popc(left[d]);
            x[d] = 0.0;
        }
        if (n > kFew) {
            // many: every lane its own dims
            todo = (1u << kOwn) - 1;
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
            for (int d = 0; d < kOwn; d++) x[d] /= block;
            n = 0;
        }
        // few: four at a time, eight lanes a dim, a lane every eighth token
        for (; n > 0; n -= 4) {
            int who = -1;                                  // the lane that has the group's dim | d << 8
#pragma unroll
            for (int g = 0; g < 4; g++) {
                int pick = -1;
#pragma unroll
                for (int d = 0; d < kOwn; d++) {
                    if (pick < 0 && left[d]) {
                        pick = (__ffs(left[d]) - 1) | d << 8;
                        left[d] &= left[d] - 1;
                    }
                }
                if (lane >> 3 == g) who = pick;
            }
            const int dim = __shfl_sync(0xffffffffu, own, who & 31) + (who >> 8);
            double y = 0.0;
            if (who >= 0) {
                const uint8_t *k0 = k_cache + t0 * D + dim;
#pragma unroll 8
                for (int t = lane & 7; t < block; t += 8)
                    y = fma((double)e4m3_to_f32(k0[(int64_t)t * D]), (double)k_scale[t0 + t], y);
            }
            __syncwarp();
#pragma unroll
            for (int m = 4; m > 0; m >>= 1) y += __shfl_xor_sync(0xffffffffu, y, m);
            y /= block;
#pragma unroll
            for (int g = 0; g < 4; g++) {
                const int to = __shfl_sync(0xffffffffu, who, 8 * g);
                const double z = __shfl_sync(0xffffffffu, y, 8 * g);
#pragma unroll
                for (int d = 0; d < kOwn; d++)
                    if (to == (lane | d << 8)) x[d] = z;
            }
        }
#pragma unroll
        for (int d = 0; d < kOwn; d++) top = fmax(top, fabs(x[d]));
#pragma unroll
        for (int m = 16; m > 0; m >>= 1) top = fmax(top, __shfl_xor_sync(0xffffffffu, top, m));
        const double exact = fmax(top, (double)1e-4f) / 448.0;
        sc = __double2float_rn(exact);
#pragma unroll
        for (int d = 0; d < kOwn; d++) {
            if (todo >> d & 1) codes = (codes & ~(0xFFu << (8 * d))) | (e4m3x2_rn_sat(f32_odd(x[d] / exact), 0.f) & 0xFF) << (8 * d);
        }
    }
    uint8_t *dst = blk_cache + (b * n_max + e) * D + own;
    if constexpr (kOwn == 4)
        *reinterpret_cast<uint32_t *>(dst) = codes;
    else
        *reinterpret_cast<uint16_t *>(dst) = (uint16_t)codes;
    if (lane == 0) blk_scale[b * n_max + e] = sc;
}

}  // namespace
}  // namespace dsa

extern "C" dsa_status dsa_block_keys(const uint8_t *k_cache, const float *k_scale, int64_t t_max, int B,
                                     int64_t start_pos, int64_t S, int D, int block, uint8_t *blk_cache,
                                     float *blk_scale, int64_t n_max, dsa_stream_t stream) {
    if (B < 0 || S < 0 || start_pos < 0 || block < 1 || n_max < 0 || t_max < 0) return DSA_ERR_INVALID_ARG;
    if (D != 64 && D != 128) return DSA_ERR_UNSUPPORTED;
    // (the kernel counts a block's tokens in 32 bits, sixteen loads ahead, and the
    // error's bound has room for the roundings of this many)
    if (block > 1 << 20) return DSA_ERR_UNSUPPORTED;
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
