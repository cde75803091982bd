// latent_rows.cuh -- the latent cache's row formats, seen from the device.
//
//   DSA_BF16        [dc bf16 | dr bf16]
//   DSA_FP8_LATENT  [dc e4m3 codes | dc/128 fp32 scales | dr bf16]
//   DSA_Q4_LATENT   [dc/2 code bytes | dr bf16 | dc/32 bf16 scales | zeros up
//                   to a multiple of 16 bytes]
// The 4-bit codes are 8 + n with n in [-7, 7], one bf16 scale s per 32 values;
// in each 32-bit word of eight codes value 2i is nibble i and value 2i + 1
// nibble i + 4, so that one shift and one mask give two neighbouring values in
// the two halves of a word.  The value a code stands for is n * s, rounded to
// bf16 like every decoded value of the library.  Codes come first so that each
// group of 32 is one aligned 16-byte piece, and the 16-byte row pitch keeps
// every piece of the row aligned.
#pragma once

#include "common.cuh"

namespace dsa {

template <int F>
__host__ __device__ constexpr int latent_rope_at(int dc) {
    return F == DSA_BF16 ? 2 * dc : F == DSA_FP8_LATENT ? dc + dc / 32 : dc / 2;
}
__host__ __device__ constexpr int latent_q4_scales_at(int dc, int dr) { return dc / 2 + 2 * dr; }

__host__ __device__ constexpr int64_t latent_fmt_row_bytes(int fmt, int dc, int dr) {
    return fmt == DSA_BF16         ? 2 * (int64_t)(dc + dr)
           : fmt == DSA_FP8_LATENT ? (int64_t)dc + dc / 32 + 2 * dr
                                   : ((int64_t)dc / 2 + 2 * dr + dc / 16 + 15) / 16 * 16;
}

// The shapes of the quantised formats; the operators over all three formats
// take the same ones for bf16 rows.
inline bool latent_shape_ok(int dc, int dr) {
    return dc >= 128 && dc <= 512 && dc % 128 == 0 && dr >= 0 && dr <= 64 && dr % 8 == 0;
}

__device__ __forceinline__ uint32_t bf16x2_bits(__nv_bfloat162 v) {
    return *reinterpret_cast<const uint32_t *>(&v);
}

// Two 4-bit codes (a word masked with 0x000F000F) times the scale pair, as
// bf16: or-ing 0x4300 makes each half the bf16 number 128 + code; subtracting
// 136 is exact (integers up to 143 have eight significand bits) and leaves n,
// and the product is rounded once.
__device__ __forceinline__ uint32_t q4_pair(uint32_t codes, __nv_bfloat162 scale) {
    const uint32_t biased = codes | 0x43004300u;
    const uint32_t offset = 0x43084308u;                    // 136, twice
    const __nv_bfloat162 n = __hsub2(*reinterpret_cast<const __nv_bfloat162 *>(&biased),
                                     *reinterpret_cast<const __nv_bfloat162 *>(&offset));
    return bf16x2_bits(__hmul2(n, scale));
}

// The eight values of one word of codes, as four bf16 pairs in order.
__device__ __forceinline__ uint4 q4_decode8(uint32_t w, __nv_bfloat162 scale) {
    return make_uint4(q4_pair(w & 0x000F000Fu, scale), q4_pair((w >> 4) & 0x000F000Fu, scale),
                      q4_pair((w >> 8) & 0x000F000Fu, scale), q4_pair((w >> 12) & 0x000F000Fu, scale));
}

// Eight e4m3 codes (two words) times the block scale, rounded to bf16 pairs.
__device__ __forceinline__ uint4 fp8_decode8(uint32_t w0, uint32_t w1, float sc) {
    uint32_t o[4];
    const uint32_t w[2] = {w0, w1};
#pragma unroll
    for (int q = 0; q < 2; q++) {
#pragma unroll
        for (int h = 0; h < 2; h++) {
            const __half2_raw hr = __nv_cvt_fp8x2_to_halfraw2(
                static_cast<__nv_fp8x2_storage_t>((w[q] >> (16 * h)) & 0xFFFFu), __NV_E4M3);
            const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&hr));
            o[2 * q + h] = bf16x2_bits(__floats2bfloat162_rn(f.x * sc, f.y * sc));
        }
    }
    return make_uint4(o[0], o[1], o[2], o[3]);
}

__device__ __forceinline__ float2 bf16x2_to_f32(uint32_t w) {
    return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
}

}  // namespace dsa
