// latent_cache.cu -- writing latent rows into a bf16, FP8 or 4-bit cache from
// the projection's output (RMS norm, rotary embedding, quantisation, append)
// and reading them back.
//
// Pages: the MLA excerpts ("DeepSeek-V3.2-Exp - Causal mask": kv_norm over the
// kv_lora_rank part of wkv_a's output and apply_rotary_emb over k_pe, before
// the cache write) and the diagram "DeepSeek Sparse Attention, one decode step
// in one layer (V3.2 sizes)" (the FP8 row).
//
// Both kernels move bytes.  The bytes of a row (1152 read and 416 written from
// bf16 to 4 bits) leave about 270 warp instructions at the memory's rate, so
// in the prologue half a warp owns a row and a lane 32 consecutive latent values,
// one 4-bit group: the group's maximum and scale need no exchange and are worked
// out once per 32 values, the codes leave as one 16-byte store, arithmetic is
// packed in pairs, a word of codes is put together by multiply-adds on the bits
// of the rounded quotients, and the next row is loaded ahead.  65536 rows with norm
// and rotation take 27.5 us from bf16 to 4 bits (257 warp instructions a row, 62% of
// the issue slots), 25.1 to FP8, 38.0 to bf16.  The read has a warp per row and eight
// values a lane, so that its wide stores are whole lines.
//
// Rounding.  What is stored is the rounding of the exact value (of the products
// and the norm taken in 64 bits): the fp32 result is used where its error leaves
// the rounded value in no doubt, and a row (or a rotary pair) where it might not,
// about sixteen 4-bit rows in a thousand, is taken again in 64 bits.  bf16 numbers
// and 4-bit scales are rounded to fp32 first, then to bf16, like every cast of an
// fp32 result.  (FP8 codes of a normed row are rounded from fp32.)
#include <algorithm>

#include "latent_rows.cuh"
#include "quant.cuh"

namespace dsa {
namespace {

constexpr int kWarps = 8;
constexpr int kSlots = 2;      // the read's chunks of eight latent values a lane: dc <= 512
constexpr int kProWarps = 4;   // warps per prologue block (four blocks an SM: registers for a row ahead)
constexpr int kProBlocks = 4;
constexpr int kVals = 32;      // the prologue's latent values a lane: half a warp holds dc <= 512

struct PrologueArgs {
    const void *kv;
    int64_t batch_stride, token_stride;      // elements
    const float *norm_w;
    float eps;
    const float *rope_cs;
    int interleaved;
    int64_t start_pos, t_max;
    uint8_t *cache;
    int64_t rows;
    int S, dc, dr;
};

// A row number as (sequence, token of n): stepped without a division per row.
template <typename I>
struct RowPos {
    I b, s, step_b, step_s, n;
    __device__ RowPos(int64_t row, int64_t step, I n) : n(n) {
        b = (I)(row / n);
        s = (I)(row - (int64_t)b * n);
        step_b = (I)(step / n);
        step_s = (I)(step - (int64_t)step_b * n);
    }
    __device__ void next() {
        b += step_b;
        // (s < n and step_s < n; the sum may pass the type's range)
        const bool over = s >= n - step_s;
        s = over ? s - (n - step_s) : s + step_s;
        b += over;
    }
};

// A lane's 32 latent values and four rotary ones as they lie in memory.
template <typename T> struct RawRow;
template <> struct RawRow<__nv_bfloat16> {
    using Vec = uint4;
    using Pair = uint32_t;
    uint4 c[4];
    uint32_t pe[2];
};
template <> struct RawRow<float> {
    using Vec = float4;
    using Pair = float2;
    float4 c[8];
    float2 pe[2];
};

__device__ __forceinline__ void widen(const RawRow<__nv_bfloat16> &r, float2 (&x)[kVals / 2], float2 (&pe)[2]) {
#pragma unroll
    for (int i = 0; i < 4; i++) {
        x[4 * i] = bf16x2_to_f32(r.c[i].x);
        x[4 * i + 1] = bf16x2_to_f32(r.c[i].y);
        x[4 * i + 2] = bf16x2_to_f32(r.c[i].z);
        x[4 * i + 3] = bf16x2_to_f32(r.c[i].w);
    }
    pe[0] = bf16x2_to_f32(r.pe[0]);
    pe[1] = bf16x2_to_f32(r.pe[1]);
}
__device__ __forceinline__ void widen(const RawRow<float> &r, float2 (&x)[kVals / 2], float2 (&pe)[2]) {
#pragma unroll
    for (int i = 0; i < 8; i++) {
        x[2 * i] = make_float2(r.c[i].x, r.c[i].y);
        x[2 * i + 1] = make_float2(r.c[i].z, r.c[i].w);
    }
    pe[0] = r.pe[0];
    pe[1] = r.pe[1];
}

// The larger of a and b, a NaN passing through: a 4-bit group that holds one gets
// a NaN scale, so that what it stands for is NaN (an FP8 code has its own NaN)
__device__ __forceinline__ float max_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ float2 splat(float x) { return make_float2(x, x); }

// The 4-bit word of eight quotients: adding 1.5 * 2^23 + 8 rounds each to the
// nearest integer n (ties to even) and leaves n + 8 in the low bits on top of a
// constant, which the sum of the shifted words carries off.
constexpr float kMagic = 12582912.f + 8.f;
constexpr uint32_t kMagicBits = 0x4B400000u;        // of 1.5 * 2^23
__device__ __forceinline__ uint32_t q4_word(const float2 *r) {          // four pairs of quotients + kMagic
    uint32_t w = 0u - kMagicBits * 0x11111111u;
#pragma unroll
    for (int i = 0; i < 4; i++) {
        w += __float_as_uint(r[i].x) << (4 * i);
        w += __float_as_uint(r[i].y) << (4 * (i + 4));
    }
    return w;
}

// A latent row's rounding in 64 bits, by the whole warp: lane = values 16 lane ..
// 16 lane + 15, half a 4-bit group.  It runs for few rows; a function of its own
// keeps its registers out of the common path.  (With the group over a warp's lanes
// its exchanges took 6.5 us a row.)
template <int F, typename T>
__device__ __noinline__ void exact_row(const T *src, uint8_t *dst, const float *w, float eps, int dc, int dr) {
    const int lane = threadIdx.x & 31;
    const bool on = 16 * lane < dc;
    float2 f[8];
#pragma unroll
    for (int i = 0; i < 8; i++) f[i] = splat(0.f);
    if (on) {
        if constexpr (sizeof(T) == 2) {
#pragma unroll
            for (int i = 0; i < 2; i++) {
                const uint4 c = reinterpret_cast<const uint4 *>(src + 16 * lane)[i];
                f[4 * i] = bf16x2_to_f32(c.x);
                f[4 * i + 1] = bf16x2_to_f32(c.y);
                f[4 * i + 2] = bf16x2_to_f32(c.z);
                f[4 * i + 3] = bf16x2_to_f32(c.w);
            }
        } else {
#pragma unroll
            for (int i = 0; i < 4; i++) {
                const float4 c = reinterpret_cast<const float4 *>(src + 16 * lane)[i];
                f[2 * i] = make_float2(c.x, c.y);
                f[2 * i + 1] = make_float2(c.z, c.w);
            }
        }
    }
    double y[16], s0 = 0.0, s1 = 0.0;
#pragma unroll
    for (int i = 0; i < 8; i++) {
        y[2 * i] = (double)f[i].x;
        y[2 * i + 1] = (double)f[i].y;
        s0 = fma(y[2 * i], y[2 * i], s0);
        s1 = fma(y[2 * i + 1], y[2 * i + 1], s1);
    }
    s0 += s1;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s0 += __shfl_xor_sync(0xffffffffu, s0, o);
    const double r = 1.0 / sqrt(s0 / dc + (double)eps);
    double amax = 0.0;
    bool nan = false;
#pragma unroll
    for (int i = 0; i < 4; i++) {
        const float4 wv = reinterpret_cast<const float4 *>(w)[on ? 4 * lane + i : 0];
        const float wf[4] = {wv.x, wv.y, wv.z, wv.w};
#pragma unroll
        for (int e = 0; e < 4; e++) {
            y[4 * i + e] = y[4 * i + e] * r * (double)wf[e];
            amax = fmax(amax, fabs(y[4 * i + e]));
            nan |= y[4 * i + e] != y[4 * i + e];
        }
    }
    if constexpr (F == DSA_Q4_LATENT) {
        amax = fmax(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
        const uint32_t bad = __ballot_sync(0xffffffffu, nan);
        float sf = __double2float_rn(fmax(amax, (double)1e-4f) / 7.0);
        if (bad >> (lane & 30) & 3) sf = __int_as_float(0x7FC00000);       // a NaN makes the group NaN
        const __nv_bfloat16 sb = __float2bfloat16_rn(sf);
        const double inv = 1.0 / (double)__bfloat162float(sb);
        uint32_t c[2] = {0, 0};
#pragma unroll
        for (int v = 0; v < 16; v++)
            c[v >> 3] |= (uint32_t)(8 + max(-7, min(7, __double2int_rn(y[v] * inv)))) << (4 * ((v & 7) / 2 + 4 * (v & 1)));
        if (on) reinterpret_cast<uint2 *>(dst)[lane] = make_uint2(c[0], c[1]);
        if (on && (lane & 1) == 0)
            reinterpret_cast<__nv_bfloat16 *>(dst + latent_q4_scales_at(dc, dr))[lane >> 1] = sb;
    } else {
        uint32_t c[8];
#pragma unroll
        for (int i = 0; i < 8; i++)
            c[i] = bf16x2_bits(__floats2bfloat162_rn(__double2float_rn(y[2 * i]), __double2float_rn(y[2 * i + 1])));
        if (on) {
            reinterpret_cast<uint4 *>(dst)[2 * lane] = make_uint4(c[0], c[1], c[2], c[3]);
            reinterpret_cast<uint4 *>(dst)[2 * lane + 1] = make_uint4(c[4], c[5], c[6], c[7]);
        }
    }
}

// The rotation of one pair (re, im) by (cos, sin), as bf16.
__device__ __forceinline__ __nv_bfloat162 rotate_bf16(float re, float im, float2 cs) {
    const float a = re * cs.x, b = im * cs.y, c = re * cs.y, d = im * cs.x;
    const float y0 = a - b, y1 = c + d;
    // three roundings each, of terms this large
    const float e0 = (fabsf(a) + fabsf(b)) * 0x1p-22f, e1 = (fabsf(c) + fabsf(d)) * 0x1p-22f;
    const __nv_bfloat162 lo = __floats2bfloat162_rn(y0 - e0, y1 - e1), hi = __floats2bfloat162_rn(y0 + e0, y1 + e1);
    if (bf16x2_bits(lo) == bf16x2_bits(hi)) return lo;
    const double z0 = (double)re * cs.x - (double)im * cs.y, z1 = (double)re * cs.y + (double)im * cs.x;
    return __floats2bfloat162_rn(__double2float_rn(z0), __double2float_rn(z1));
}

// Row r = (b, s): y = c * rsqrt(mean(c^2) + eps) * w (without norm_w, y = c),
// k_pe times the position's (cos, sin), then the format's rounding.  (Without a
// norm nothing is rounded from 64 bits, and the registers around that call are free.)
template <int F, typename T, bool norm>
__global__ void __launch_bounds__(32 * kProWarps, kProBlocks) latent_prologue_kernel(const PrologueArgs a) {
    // the norm's weights, a lane's 32 at a pitch that keeps lanes off each
    // other's banks
    constexpr int kPitch = kVals + 4;
    __shared__ float4 w_sm[16 * kPitch / 4], w_flat[512 / 4];
    const int lane = threadIdx.x & 31, l16 = lane & 15;
    static_assert(32 * kProWarps >= 512 / 4, "one load fills the weights");
    bool far_out = false;          // weights with which products could leave fp32's range
    if (norm && threadIdx.x < a.dc / 4) {
        const float4 v = reinterpret_cast<const float4 *>(a.norm_w)[threadIdx.x];
        w_flat[threadIdx.x] = v;
        w_sm[(threadIdx.x / 8) * (kPitch / 4) + threadIdx.x % 8] = v;
        const float top = fmaxf(fmaxf(fabsf(v.x), fabsf(v.y)), fmaxf(fabsf(v.z), fabsf(v.w)));
        auto small = [](float x) { return x != 0.f && fabsf(x) < 0x1p-60f; };
        far_out = top > 0x1p60f || small(v.x) || small(v.y) || small(v.z) || small(v.w);
    }
    far_out = __syncthreads_or(far_out);
    const int64_t rb = latent_fmt_row_bytes(F, a.dc, a.dr);
    const float inv_dc = 1.f / (float)a.dc;
    const double inv_dc64 = 1.0 / a.dc;
    const bool has_c = kVals * l16 < a.dc;
    // rotary pairs 2 l and 2 l + 1: elements 4 l .. 4 l + 3, or, when the
    // embedding is not interleaved, 2 l, 2 l + 1 and those dr/2 further on
    const int half = a.dr / 2;
    const bool has_pe = 4 * l16 < a.dr, halves = a.rope_cs && !a.interleaved;
    const int e0 = halves ? 2 * l16 : 4 * l16, e1 = halves ? 2 * l16 + half : 4 * l16 + 2;

    RawRow<T> raw = {};
    float4 cs = make_float4(1.f, 0.f, 1.f, 0.f);
    auto source = [&](int b, int s) {
        return static_cast<const T *>(a.kv) + b * a.batch_stride + s * a.token_stride;
    };
    auto fetch = [&](int b, int s) {
        const T *src = source(b, s);
        if (has_c) {
            constexpr int n = sizeof(raw.c) / 16;
#pragma unroll
            for (int i = 0; i < n; i++) raw.c[i] = reinterpret_cast<const typename RawRow<T>::Vec *>(src + kVals * l16)[i];
        }
        if (has_pe) {
            raw.pe[0] = *reinterpret_cast<const typename RawRow<T>::Pair *>(src + a.dc + e0);
            raw.pe[1] = *reinterpret_cast<const typename RawRow<T>::Pair *>(src + a.dc + e1);
            if (a.rope_cs) cs = reinterpret_cast<const float4 *>(a.rope_cs + (int64_t)s * a.dr)[l16];
        }
    };
    // a warp's two rows: 2 k and 2 k + 1
    const int64_t step = 2 * (int64_t)gridDim.x * kProWarps;
    int64_t r = 2 * ((int64_t)blockIdx.x * kProWarps + (threadIdx.x >> 5)) + (lane >> 4);
    RowPos<int> at(r, step, a.S);
    if (r < a.rows) fetch(at.b, at.s);
    for (; r - (lane >> 4) < a.rows; r += step) {
        const bool on = r < a.rows;
        const int b = at.b, s = at.s;
        uint8_t *dst = a.cache + (b * a.t_max + a.start_pos + s) * rb;
        float2 x[kVals / 2], pe[2];
        widen(raw, x, pe);
        const float4 cs_now = cs;
        at.next();
        if (r + step < a.rows) fetch(at.b, at.s);

        float rms = 1.f;
        bool doubt = false;
        if constexpr (norm) {
            // What fp32 may be off by, with u = 2^-24: the sum's chains of eight, two
            // and four steps and the mean 16 u, so the root 8 u and 2 u of its own; a
            // product u each.  bf16 values, where every one of a row's 512 is next to
            // a border now and then, take the sum and the root in 64 bits.
            if constexpr (F == DSA_BF16) {
                double s0 = 0.0, s1 = 0.0;
#pragma unroll
                for (int e = 0; e < kVals / 2; e++) {
                    s0 = fma((double)x[e].x, (double)x[e].x, s0);
                    s1 = fma((double)x[e].y, (double)x[e].y, s1);
                }
                s0 += s1;
#pragma unroll
                for (int m = 8; m > 0; m >>= 1) s0 += __shfl_xor_sync(0xffffffffu, s0, m);
                const double v = fma(s0, inv_dc64, (double)a.eps);
                const float vf = (float)v;
                doubt = far_out || !(vf > 0x1p-80f && vf < 0x1p80f);       // squares that fp32 cannot hold
                const double r0 = (double)rsqrtf(vf);
                rms = (float)fma(r0 * 0.5, fma(-v * r0, r0, 1.0), r0);     // a Newton step
            } else {
                const auto mean_square = [&](float eps) {  // of the half warp's row, plus eps
                    float2 s0 = make_float2(0.f, 0.f), s1 = s0;
#pragma unroll
                    for (int e = 0; e < kVals / 2; e += 2) {
                        s0 = __ffma2_rn(x[e], x[e], s0);
                        s1 = __ffma2_rn(x[e + 1], x[e + 1], s1);
                    }
                    float ss = (s0.x + s0.y) + (s1.x + s1.y);
#pragma unroll
                    for (int m = 8; m > 0; m >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, m);
                    return fmaf(ss, inv_dc, eps);
                };
                float v = mean_square(a.eps);
                doubt = !(v > 0x1p-80f && v < 0x1p80f);    // squares that fp32 cannot hold
                if constexpr (F == DSA_FP8_LATENT) {
                    // such a row is taken times a power of two, which the norm takes
                    // out again (4-bit rows are rounded from 64-bit sums below)
                    if (__any_sync(0xffffffffu, doubt)) {
                        const float k = !doubt ? 1.f : v < 1.f ? 0x1p90f : 0x1p-80f;
#pragma unroll
                        for (int e = 0; e < kVals / 2; e++) x[e] = __fmul2_rn(x[e], splat(k));
                        v = mean_square(a.eps * k * k);
                    }
                } else {
                    doubt |= far_out;
                }
                rms = rsqrtf(v);
                if (rms != 0.f) rms = fmaf(rms * 0.5f, fmaf(-v * rms, rms, 1.f), rms);      // a Newton step: within a rounding or two
#pragma unroll
                for (int e = 0; e < kVals / 4; e++) {
                    const float4 wv = w_sm[l16 * (kPitch / 4) + e];
                    // the norm's factor comes later
                    x[2 * e] = __fmul2_rn(x[2 * e], make_float2(wv.x, wv.y));
                    x[2 * e + 1] = __fmul2_rn(x[2 * e + 1], make_float2(wv.z, wv.w));
                }
            }
        }
        if constexpr (F == DSA_BF16) {
#pragma unroll
            for (int i = 0; i < 4; i++) {
                uint32_t c[4];
#pragma unroll
                for (int e = 0; e < 4; e++) {
                    const float4 wv = norm ? w_sm[l16 * (kPitch / 4) + 2 * i + e / 2] : make_float4(1.f, 1.f, 1.f, 1.f);
                    // (weight times root stays in range whatever x is)
                    const float2 y = __fmul2_rn(x[4 * i + e], __fmul2_rn(e & 1 ? make_float2(wv.z, wv.w) : make_float2(wv.x, wv.y), splat(rms)));
                    c[e] = bf16x2_bits(__floats2bfloat162_rn(y.x, y.y));
                    // three roundings, less than three of the 2^16 units below bf16: in
                    // doubt within four units of the middle
                    doubt |= ((__float_as_uint(y.x) + 0x8004u) & 0xFFFFu) <= 8u || ((__float_as_uint(y.y) + 0x8004u) & 0xFFFFu) <= 8u;
                }
                if (on && has_c) reinterpret_cast<uint4 *>(dst)[4 * l16 + i] = make_uint4(c[0], c[1], c[2], c[3]);
            }
        } else {
            float amax = 0.f;
            if constexpr (F == DSA_FP8_LATENT) {
#pragma unroll
                for (int e = 0; e < kVals / 2; e++) amax = fmaxf(amax, fmaxf(fabsf(x[e].x), fabsf(x[e].y)));
                // a block of 128 is four lanes'
                amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
                amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
                const float sc = div_rn_by(fmaxf(amax * rms, 1e-4f), 448.0f, 1.0f / 448.0f), rs = __frcp_rn(sc);
                const float2 rs2 = splat(rs), ns2 = splat(-sc);
                uint32_t words[kVals / 4];
#pragma unroll
                for (int i = 0; i < kVals / 4; i++) {
                    uint32_t c[2];
#pragma unroll
                    for (int e = 0; e < 2; e++) {          // the correctly rounded quotient (div_rn_by, in pairs)
                        const float2 y = __fmul2_rn(x[2 * i + e], splat(rms));
                        const float2 q0 = __fmul2_rn(y, rs2);
                        const float2 q = __ffma2_rn(__ffma2_rn(q0, ns2, y), rs2, q0);
                        c[e] = e4m3x2_rn_sat(q.x, q.y);
                    }
                    words[i] = c[0] | c[1] << 16;
                }
                if (on && has_c) {
                    if ((rb & 15) == 0) {
                        reinterpret_cast<uint4 *>(dst)[2 * l16] = make_uint4(words[0], words[1], words[2], words[3]);
                        reinterpret_cast<uint4 *>(dst)[2 * l16 + 1] = make_uint4(words[4], words[5], words[6], words[7]);
                    } else {                   // (rows of shapes other than 512 are only 4-byte aligned)
#pragma unroll
                        for (int i = 0; i < kVals / 4; i++) reinterpret_cast<uint32_t *>(dst)[8 * l16 + i] = words[i];
                    }
                }
                if (on && has_c && (l16 & 3) == 0) reinterpret_cast<float *>(dst + a.dc)[l16 >> 2] = sc;
            } else {
#pragma unroll
                for (int e = 0; e < kVals / 2; e++) amax = max_nan(amax, max_nan(fabsf(x[e].x), fabsf(x[e].y)));
                const float st = div_rn_by(max_nan(amax * rms, 1e-4f), 7.0f, 1.0f / 7.0f);
                const __nv_bfloat16 sb = __float2bfloat16_rn(st);
                const float sc = __bfloat162float(sb), rs = __frcp_rn(sc);
                if constexpr (norm) {
                    // in doubt: a quotient, off by 14 u of itself (weight, root, the
                    // scale's reciprocal, two products), which is 2^-17.3 at seven,
                    // within 2^-17 of a border; a scale, off by 13 u or fewer than 13
                    // of the 2^16 units below bf16, within 16 units of the middle
                    const float2 k = splat(rms * rs);
                    float far = 0.f;
#pragma unroll
                    for (int e = 0; e < kVals / 2; e++) {
                        const float2 q = __fmul2_rn(x[e], k);
                        x[e] = __fadd2_rn(q, splat(kMagic));
                        const float2 n = __fadd2_rn(x[e], splat(-kMagic));
                        const float2 d = __ffma2_rn(q, splat(-1.f), n);
                        far = fmaxf(far, fmaxf(fabsf(d.x), fabsf(d.y)));
                    }
                    doubt |= far > 0.5f - 0x1p-17f || ((__float_as_uint(st) + 0x8010u) & 0xFFFFu) <= 32u;
                } else {
                    const float2 rs2 = splat(rs), ns2 = splat(-sc);
#pragma unroll
                    for (int e = 0; e < kVals / 2; e++) {  // the correctly rounded quotient
                        const float2 q0 = __fmul2_rn(x[e], rs2);
                        x[e] = __fadd2_rn(__ffma2_rn(__ffma2_rn(q0, ns2, x[e]), rs2, q0), splat(kMagic));
                    }
                }
                if (on && has_c) {
                    reinterpret_cast<uint4 *>(dst)[l16] = make_uint4(q4_word(x), q4_word(x + 4), q4_word(x + 8), q4_word(x + 12));
                    reinterpret_cast<__nv_bfloat16 *>(dst + latent_q4_scales_at(a.dc, a.dr))[l16] = sb;
                }
            }
        }
        if constexpr (F != DSA_FP8_LATENT && norm) {
            const uint32_t rows = __ballot_sync(0xffffffffu, doubt && on && has_c);
            if (rows) {
                __syncwarp();                              // the fp32 result's stores come first
#pragma unroll 1
                for (int h = 0; h < 2; h++) {
                    if (!(rows >> (16 * h) & 0xFFFFu)) continue;
                    const int hb = __shfl_sync(0xffffffffu, b, 16 * h), hs = __shfl_sync(0xffffffffu, s, 16 * h);
                    exact_row<F, T>(source(hb, hs), a.cache + (hb * a.t_max + a.start_pos + hs) * rb,
                                    reinterpret_cast<const float *>(w_flat), a.eps, a.dc, a.dr);
                }
            }
        }
        if (on && has_pe) {
            __nv_bfloat162 *out = reinterpret_cast<__nv_bfloat162 *>(dst + latent_rope_at<F>(a.dc));
            if (halves) {
                const __nv_bfloat162 y0 = rotate_bf16(pe[0].x, pe[1].x, make_float2(cs_now.x, cs_now.y));
                const __nv_bfloat162 y1 = rotate_bf16(pe[0].y, pe[1].y, make_float2(cs_now.z, cs_now.w));
                out[e0 / 2] = __halves2bfloat162(y0.x, y1.x);
                out[e1 / 2] = __halves2bfloat162(y0.y, y1.y);
            } else {
                out[e0 / 2] = a.rope_cs ? rotate_bf16(pe[0].x, pe[0].y, make_float2(cs_now.x, cs_now.y)) : __floats2bfloat162_rn(pe[0].x, pe[0].y);
                out[e1 / 2] = a.rope_cs ? rotate_bf16(pe[1].x, pe[1].y, make_float2(cs_now.z, cs_now.w)) : __floats2bfloat162_rn(pe[1].x, pe[1].y);
            }
        }
        if (F == DSA_Q4_LATENT) {              // the row's end: zeros up to its pitch
            const int end = latent_q4_scales_at(a.dc, a.dr) + a.dc / 16 + 2 * l16;
            if (on && end < rb) *reinterpret_cast<uint16_t *>(dst + end) = 0;
        }
    }
}

// A lane's share of a row as it lies in the cache, and its values.
template <int F> struct RawRead;
template <> struct RawRead<DSA_BF16> { uint4 c[kSlots]; };
template <> struct RawRead<DSA_FP8_LATENT> { uint2 c[kSlots]; float s[kSlots]; };
template <> struct RawRead<DSA_Q4_LATENT> { uint32_t c[kSlots]; __nv_bfloat16 s[kSlots]; };

template <int F>
__device__ __forceinline__ void read_raw(RawRead<F> &r, const uint8_t *row, int u, int chunk, int dc, int dr) {
    if constexpr (F == DSA_BF16) {
        r.c[u] = reinterpret_cast<const uint4 *>(row)[chunk];
    } else if constexpr (F == DSA_FP8_LATENT) {
        // (rows of some shapes are only 4-byte aligned)
        const uint32_t *c = reinterpret_cast<const uint32_t *>(row) + 2 * chunk;
        r.c[u] = make_uint2(c[0], c[1]);
        r.s[u] = *reinterpret_cast<const float *>(row + dc + 4 * (chunk >> 4));
    } else {
        r.c[u] = reinterpret_cast<const uint32_t *>(row)[chunk];
        r.s[u] = *reinterpret_cast<const __nv_bfloat16 *>(row + latent_q4_scales_at(dc, dr) + 2 * (chunk >> 2));
    }
}
template <int F>
__device__ __forceinline__ uint4 read_values(const RawRead<F> &r, int u) {
    if constexpr (F == DSA_BF16)
        return r.c[u];
    else if constexpr (F == DSA_FP8_LATENT)
        return fp8_decode8(r.c[u].x, r.c[u].y, r.s[u]);
    else
        return q4_decode8(r.c[u], __halves2bfloat162(r.s[u], r.s[u]));
}

// Row i of the output = cache row idx[i] (zeros for -1) or start_pos + i.  A
// warp takes kRows rows at a time, all their loads before the first decoding
// (an absent row's or chunk's loads go to row 0 or chunk 0 and are not used).
template <int F, typename T, int kRows>
__global__ void __launch_bounds__(32 * kWarps)
latent_read_kernel(const uint8_t *__restrict__ cache, int64_t t_max, const int32_t *__restrict__ idx,
                   int64_t start_pos, int64_t rows, int64_t n, int dc, int dr, T *__restrict__ out, int *err) {
    const int lane = threadIdx.x & 31;
    const int chunks = dc / 8;
    const int64_t rb = latent_fmt_row_bytes(F, dc, dr);
    const int64_t step = (int64_t)gridDim.x * kWarps * kRows;
    int64_t r0 = ((int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5)) * kRows;
    if (r0 >= rows) return;
    for (RowPos<int64_t> at(r0, step, n); r0 < rows; r0 += step, at.next()) {
        int64_t t[kRows], b = at.b, s = at.s;
#pragma unroll
        for (int i = 0; i < kRows; i++) {
            if (i > 0 && r0 + i < rows && ++s >= n) {      // (a row past the end is the last one again)
                s = 0;
                b++;
            }
            t[i] = idx ? (int64_t)idx[b * n + s] : start_pos + s;
            if (t[i] >= t_max && lane == 0) record_error(err, DSA_ERR_DEVICE);
            t[i] = t[i] < 0 || t[i] >= t_max ? -1 : b * t_max + t[i];
        }
        RawRead<F> raw[kRows];
        uint32_t pe[kRows];
#pragma unroll
        for (int i = 0; i < kRows; i++) {
            const uint8_t *row = cache + (t[i] < 0 ? 0 : t[i]) * rb;
#pragma unroll
            for (int u = 0; u < kSlots; u++)
                read_raw<F>(raw[i], row, u, lane + 32 * u < chunks ? lane + 32 * u : 0, dc, dr);
            pe[i] = dr ? reinterpret_cast<const uint32_t *>(row + latent_rope_at<F>(dc))[lane < dr / 2 ? lane : 0] : 0u;
        }
#pragma unroll
        for (int i = 0; i < kRows; i++) {
            if (r0 + i >= rows) break;
            T *dst = out + (r0 + i) * (dc + dr);
#pragma unroll
            for (int u = 0; u < kSlots; u++) {
                const int chunk = lane + 32 * u;
                if (chunk >= chunks) continue;
                const uint4 v = t[i] < 0 ? make_uint4(0, 0, 0, 0) : read_values<F>(raw[i], u);
                if constexpr (sizeof(T) == 2) {
                    reinterpret_cast<uint4 *>(dst)[chunk] = v;
                } else {
                    const float2 f0 = bf16x2_to_f32(v.x), f1 = bf16x2_to_f32(v.y), f2 = bf16x2_to_f32(v.z),
                                 f3 = bf16x2_to_f32(v.w);
                    reinterpret_cast<float4 *>(dst)[2 * chunk] = make_float4(f0.x, f0.y, f1.x, f1.y);
                    reinterpret_cast<float4 *>(dst)[2 * chunk + 1] = make_float4(f2.x, f2.y, f3.x, f3.y);
                }
            }
            if (lane < dr / 2) {
                const uint32_t v = t[i] < 0 ? 0u : pe[i];
                if constexpr (sizeof(T) == 2)
                    reinterpret_cast<uint32_t *>(dst + dc)[lane] = v;
                else
                    reinterpret_cast<float2 *>(dst + dc)[lane] = bf16x2_to_f32(v);
            }
        }
    }
}

// `cap` blocks per SM at most (the kernels stride over the rest)
unsigned warp_grid(int64_t rows, int cap) {
    const int64_t blocks = (rows + kWarps - 1) / kWarps, most = (int64_t)num_sms() * cap;
    return (unsigned)(blocks < most ? blocks : most);
}

template <typename T, bool norm>
void launch_prologue(dsa_dtype fmt, const PrologueArgs &a, cudaStream_t st) {
    const int64_t blocks = (a.rows + 2 * kProWarps - 1) / (2 * kProWarps);
    const unsigned grid = (unsigned)std::min<int64_t>(blocks, (int64_t)num_sms() * kProBlocks);   // each warp strides on
    if (fmt == DSA_BF16)
        latent_prologue_kernel<DSA_BF16, T, norm><<<grid, 32 * kProWarps, 0, st>>>(a);
    else if (fmt == DSA_FP8_LATENT)
        latent_prologue_kernel<DSA_FP8_LATENT, T, norm><<<grid, 32 * kProWarps, 0, st>>>(a);
    else
        latent_prologue_kernel<DSA_Q4_LATENT, T, norm><<<grid, 32 * kProWarps, 0, st>>>(a);
}

template <int F, typename T>
void launch_read_fmt(const uint8_t *cache, int64_t t_max, const int32_t *idx, int64_t start_pos, int64_t rows,
                     int64_t n, int dc, int dr, T *out, cudaStream_t st) {
    int *err = device_error_word();
    // Four rows a warp where a row's stores are few (bf16 out: 28.8 against 34.6
    // us with one at 100000 4-bit rows); one where they are not (fp32 out: 51.4
    // against 58.3 us), and where the rows do not give every resident warp four.
    if (sizeof(T) == 4 || rows <= (int64_t)num_sms() * 8 * kWarps)
        latent_read_kernel<F, T, 1><<<warp_grid(rows, 1 << 16), 32 * kWarps, 0, st>>>(cache, t_max, idx, start_pos, rows, n, dc, dr, out, err);
    else
        latent_read_kernel<F, T, 4><<<warp_grid((rows + 3) / 4, 1 << 16), 32 * kWarps, 0, st>>>(cache, t_max, idx, start_pos, rows, n, dc, dr, out, err);
}

template <typename T>
void launch_read(dsa_dtype fmt, const uint8_t *cache, int64_t t_max, const int32_t *idx, int64_t start_pos,
                 int64_t rows, int64_t n, int dc, int dr, T *out, cudaStream_t st) {
    if (fmt == DSA_BF16)
        launch_read_fmt<DSA_BF16>(cache, t_max, idx, start_pos, rows, n, dc, dr, out, st);
    else if (fmt == DSA_FP8_LATENT)
        launch_read_fmt<DSA_FP8_LATENT>(cache, t_max, idx, start_pos, rows, n, dc, dr, out, st);
    else
        launch_read_fmt<DSA_Q4_LATENT>(cache, t_max, idx, start_pos, rows, n, dc, dr, out, st);
}

}  // namespace
}  // namespace dsa

extern "C" int64_t dsa_latent_q4_row_bytes(int dc, int dr) {
    return dsa::latent_fmt_row_bytes(DSA_Q4_LATENT, dc, dr);
}

extern "C" dsa_status dsa_latent_prologue(const void *kv, dsa_dtype x_dtype, int64_t batch_stride,
                                          int64_t token_stride, int B, int S, int dc, int dr,
                                          const float *norm_w, float eps, const float *rope_cs,
                                          int interleaved, int64_t start_pos, int64_t t_max,
                                          void *cache, dsa_dtype cache_dt, dsa_stream_t stream) {
    if (B < 0 || S < 0 || start_pos < 0 || t_max < 0) return DSA_ERR_INVALID_ARG;
    if (x_dtype != DSA_F32 && x_dtype != DSA_BF16) return DSA_ERR_INVALID_ARG;
    if (cache_dt != DSA_BF16 && cache_dt != DSA_FP8_LATENT && cache_dt != DSA_Q4_LATENT)
        return DSA_ERR_INVALID_ARG;
    if (!dsa::latent_shape_ok(dc, dr)) return DSA_ERR_UNSUPPORTED;
    if (start_pos > t_max - S) return DSA_ERR_INVALID_ARG;
    if (B == 0 || S == 0) return DSA_OK;
    if (!kv || !cache) return DSA_ERR_INVALID_ARG;
    const int64_t per16 = x_dtype == DSA_BF16 ? 8 : 4;
    if ((S > 1 && token_stride < dc + dr) || (B > 1 && batch_stride < dc + dr)) return DSA_ERR_INVALID_ARG;
    if ((S > 1 && token_stride % per16) || (B > 1 && batch_stride % per16)) return DSA_ERR_INVALID_ARG;
    if (!dsa::aligned16(kv) || !dsa::aligned16(cache) || (norm_w && !dsa::aligned16(norm_w)) ||
        (rope_cs && !dsa::aligned16(rope_cs)))
        return DSA_ERR_INVALID_ARG;
    if (norm_w && !(eps >= 0.f)) return DSA_ERR_INVALID_ARG;
    dsa::PrologueArgs a = {};
    a.kv = kv;
    a.batch_stride = batch_stride;
    a.token_stride = token_stride;
    a.norm_w = norm_w;
    a.eps = eps;
    a.rope_cs = rope_cs;
    a.interleaved = interleaved;
    a.start_pos = start_pos;
    a.t_max = t_max;
    a.cache = static_cast<uint8_t *>(cache);
    a.rows = (int64_t)B * S;
    a.S = S;
    a.dc = dc;
    a.dr = dr;
    const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    if (x_dtype == DSA_BF16)
        norm_w ? dsa::launch_prologue<__nv_bfloat16, true>(cache_dt, a, st) : dsa::launch_prologue<__nv_bfloat16, false>(cache_dt, a, st);
    else
        norm_w ? dsa::launch_prologue<float, true>(cache_dt, a, st) : dsa::launch_prologue<float, false>(cache_dt, a, st);
    return dsa::launch_status();
}

extern "C" dsa_status dsa_latent_read(const void *cache, dsa_dtype cache_dt, int64_t t_max,
                                      const int32_t *idx, int64_t start_pos, int B, int64_t n,
                                      int dc, int dr, void *out, dsa_dtype out_dtype,
                                      dsa_stream_t stream) {
    if (B < 0 || n < 0 || t_max < 0 || (!idx && start_pos < 0)) return DSA_ERR_INVALID_ARG;
    if (out_dtype != DSA_F32 && out_dtype != DSA_BF16) return DSA_ERR_INVALID_ARG;
    if (cache_dt != DSA_BF16 && cache_dt != DSA_FP8_LATENT && cache_dt != DSA_Q4_LATENT)
        return DSA_ERR_INVALID_ARG;
    if (!dsa::latent_shape_ok(dc, dr)) return DSA_ERR_UNSUPPORTED;
    if (!idx && start_pos > t_max - n) return DSA_ERR_INVALID_ARG;
    if (B == 0 || n == 0) return DSA_OK;
    if (t_max == 0 || n > INT64_MAX / B) return DSA_ERR_INVALID_ARG;     // no row to name; no such output
    if (!cache || !out || !dsa::aligned16(cache) || !dsa::aligned16(out) ||
        (reinterpret_cast<uintptr_t>(idx) & 3))
        return DSA_ERR_INVALID_ARG;
    const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    const uint8_t *c = static_cast<const uint8_t *>(cache);
    if (out_dtype == DSA_BF16)
        dsa::launch_read(cache_dt, c, t_max, idx, start_pos, B * n, n, dc, dr, static_cast<__nv_bfloat16 *>(out), st);
    else
        dsa::launch_read(cache_dt, c, t_max, idx, start_pos, B * n, n, dc, dr, static_cast<float *>(out), st);
    return dsa::launch_status();
}
