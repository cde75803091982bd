// latent_cache.cu -- writing latent rows into a bf16, FP8 or 4-bit cache from
// the projection's output (RMS norm, rotary embedding, quantisation, append)
// and reading them back.
//
// Pages: the MLA excerpts ("DeepSeek-V3.2-Exp - Causal mask": kv_norm over the
// kv_lora_rank part of wkv_a's output and apply_rotary_emb over k_pe, before
// the cache write) and the diagram "DeepSeek Sparse Attention, one decode step
// in one layer (V3.2 sizes)" (the FP8 row).
//
// Both kernels move bytes: a warp owns a row, a lane eight consecutive latent
// values at a time (one 16-byte bf16 load, one word of 4-bit codes), so that a
// row's loads and stores are whole lines, and four lanes hold a 4-bit group,
// sixteen an FP8 block: their maxima are two or four shuffles.
#include "latent_rows.cuh"
#include "quant.cuh"

namespace dsa {
namespace {

constexpr int kWarps = 8;
constexpr int kSlots = 2;      // chunks of eight latent values a lane may hold: dc <= 512

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

template <typename T>
__device__ __forceinline__ void load8(const T *p, float (&v)[8]) {
    if constexpr (sizeof(T) == 2) {
        const uint4 w = *reinterpret_cast<const uint4 *>(p);
        const uint32_t ws[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int i = 0; i < 4; i++) {
            const float2 f = bf16x2_to_f32(ws[i]);
            v[2 * i] = f.x;
            v[2 * i + 1] = f.y;
        }
    } else {
        const float4 a = reinterpret_cast<const float4 *>(p)[0], b = reinterpret_cast<const float4 *>(p)[1];
        v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
        v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
    }
}

// Row r = (b, s): y = c * rsqrt(mean(c^2) + eps) * w (without norm_w, y = c),
// k_pe times the position's (cos, sin), then the format's rounding.  Sums and
// products stay in fp32 until that one rounding.
template <int F, typename T>
__global__ void __launch_bounds__(32 * kWarps)
latent_prologue_kernel(const PrologueArgs a) {
    const int lane = threadIdx.x & 31;
    const int chunks = a.dc / 8;
    const int64_t rb = latent_fmt_row_bytes(F, a.dc, a.dr);
    float w[kSlots][8];
    if (a.norm_w) {
#pragma unroll
        for (int u = 0; u < kSlots; u++)
            if (lane + 32 * u < chunks) load8(a.norm_w + 8 * (lane + 32 * u), w[u]);
    }
    const int64_t step = (int64_t)gridDim.x * kWarps;
    for (int64_t r = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5); r < a.rows; r += step) {
        const int64_t b = r / a.S, s = r - b * a.S;
        const T *src = static_cast<const T *>(a.kv) + b * a.batch_stride + s * a.token_stride;
        uint8_t *dst = a.cache + (b * a.t_max + a.start_pos + s) * rb;
        float x[kSlots][8];
#pragma unroll
        for (int u = 0; u < kSlots; u++) {
            if (lane + 32 * u < chunks) {
                load8(src + 8 * (lane + 32 * u), x[u]);
            } else {
#pragma unroll
                for (int e = 0; e < 8; e++) x[u][e] = 0.f;
            }
        }
        // the rotary pair of this lane: elements (2l, 2l + 1), or (l, l + dr/2)
        // when the embedding is not interleaved
        const int half = a.dr / 2;
        const bool has_pe = lane < half;
        const bool halves = a.rope_cs && !a.interleaved;
        const int e0 = halves ? lane : 2 * lane, e1 = halves ? lane + half : 2 * lane + 1;
        float p0 = 0.f, p1 = 0.f;
        if (has_pe) {
            p0 = to_f32<T>(src[a.dc + e0]);
            p1 = to_f32<T>(src[a.dc + e1]);
            if (a.rope_cs) {
                const float2 cs = reinterpret_cast<const float2 *>(a.rope_cs)[s * half + lane];
                const float y0 = __fsub_rn(__fmul_rn(p0, cs.x), __fmul_rn(p1, cs.y));
                p1 = __fadd_rn(__fmul_rn(p0, cs.y), __fmul_rn(p1, cs.x));
                p0 = y0;
            }
        }
        if (a.norm_w) {
            float ss = 0.f;
#pragma unroll
            for (int u = 0; u < kSlots; u++)
#pragma unroll
                for (int e = 0; e < 8; e++) ss = fmaf(x[u][e], x[u][e], ss);
            const float rms = __frcp_rn(__fsqrt_rn(warp_sum(ss) / (float)a.dc + a.eps));
#pragma unroll
            for (int u = 0; u < kSlots; u++)
                if (lane + 32 * u < chunks)
#pragma unroll
                    for (int e = 0; e < 8; e++) x[u][e] = x[u][e] * rms * w[u][e];
        }
#pragma unroll
        for (int u = 0; u < kSlots; u++) {
            const int chunk = lane + 32 * u;
            if (F != DSA_BF16) {
                // (every lane takes part in the shuffles; a group lies within one u)
                float amax = 0.f;
#pragma unroll
                for (int e = 0; e < 8; e++) amax = fmaxf(amax, fabsf(x[u][e]));
#pragma unroll
                for (int m = 1; m < (F == DSA_FP8_LATENT ? 16 : 4); m <<= 1)
                    amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, m));
                amax = fmaxf(amax, 1e-4f);
                if (chunk < chunks) {
                    if constexpr (F == DSA_FP8_LATENT) {
                        const float sc = __fdiv_rn(amax, 448.0f), rs = __frcp_rn(sc);
                        uint32_t c[4];
#pragma unroll
                        for (int e = 0; e < 4; e++)
                            c[e] = e4m3x2_rn_sat(div_rn_by(x[u][2 * e], sc, rs), div_rn_by(x[u][2 * e + 1], sc, rs));
                        // (rows of some shapes are only 4-byte aligned)
                        reinterpret_cast<uint32_t *>(dst)[2 * chunk] = c[0] | c[1] << 16;
                        reinterpret_cast<uint32_t *>(dst)[2 * chunk + 1] = c[2] | c[3] << 16;
                        if ((chunk & 15) == 0) reinterpret_cast<float *>(dst + a.dc)[chunk >> 4] = sc;
                    } else {
                        const __nv_bfloat16 sb = __float2bfloat16_rn(__fdiv_rn(amax, 7.0f));
                        const float sc = __bfloat162float(sb), rs = __frcp_rn(sc);
                        uint32_t c = 0;
#pragma unroll
                        for (int e = 0; e < 8; e++) {
                            const int n = max(-7, min(7, __float2int_rn(div_rn_by(x[u][e], sc, rs))));
                            c |= (uint32_t)(n + 8) << (4 * (e / 2 + 4 * (e & 1)));
                        }
                        reinterpret_cast<uint32_t *>(dst)[chunk] = c;
                        if ((chunk & 3) == 0)
                            reinterpret_cast<__nv_bfloat16 *>(dst + latent_q4_scales_at(a.dc, a.dr))[chunk >> 2] = sb;
                    }
                }
            } else if (chunk < chunks) {
                uint32_t c[4];
#pragma unroll
                for (int e = 0; e < 4; e++) c[e] = bf16x2_bits(__floats2bfloat162_rn(x[u][2 * e], x[u][2 * e + 1]));
                reinterpret_cast<uint4 *>(dst)[chunk] = make_uint4(c[0], c[1], c[2], c[3]);
            }
        }
        if (has_pe) {
            __nv_bfloat16 *pe = reinterpret_cast<__nv_bfloat16 *>(dst + latent_rope_at<F>(a.dc));
            pe[e0] = __float2bfloat16_rn(p0);
            pe[e1] = __float2bfloat16_rn(p1);
        }
        if (F == DSA_Q4_LATENT) {              // the row's end: zeros up to its pitch
            const int at = latent_q4_scales_at(a.dc, a.dr) + a.dc / 16;
            if (at + 2 * lane < rb) *reinterpret_cast<uint16_t *>(dst + at + 2 * lane) = 0;
        }
    }
}

// Row i of the output = cache row idx[i] (zeros for -1) or start_pos + i.
template <int F, typename T>
__global__ void __launch_bounds__(32 * kWarps)
latent_read_kernel(const uint8_t *__restrict__ cache, int64_t t_max, const int32_t *__restrict__ idx,
                   int64_t start_pos, int64_t rows, int64_t n, int dc, int dr, T *__restrict__ out,
                   int *err) {
    const int lane = threadIdx.x & 31;
    const int chunks = dc / 8;
    const int64_t rb = latent_fmt_row_bytes(F, dc, dr);
    const int64_t step = (int64_t)gridDim.x * kWarps;
    for (int64_t r = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5); r < rows; r += step) {
        const int64_t b = r / n;
        int64_t t = idx ? (int64_t)idx[r] : start_pos + (r - b * n);
        if (t >= t_max) {
            if (lane == 0) record_error(err, DSA_ERR_DEVICE);
            t = -1;
        }
        const uint8_t *row = cache + (b * t_max + (t < 0 ? 0 : t)) * rb;
        T *dst = out + r * (dc + dr);
#pragma unroll
        for (int u = 0; u < kSlots; u++) {
            const int chunk = lane + 32 * u;
            if (chunk >= chunks) continue;
            const uint4 v = t < 0 ? make_uint4(0, 0, 0, 0) : latent_chunk8<F>(row, dc, dr, chunk);
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
            const uint32_t v = t < 0 ? 0u : reinterpret_cast<const uint32_t *>(row + latent_rope_at<F>(dc))[lane];
            if constexpr (sizeof(T) == 2)
                reinterpret_cast<uint32_t *>(dst + dc)[lane] = v;
            else
                reinterpret_cast<float2 *>(dst + dc)[lane] = bf16x2_to_f32(v);
        }
    }
}

unsigned warp_grid(int64_t rows) {
    const int64_t blocks = (rows + kWarps - 1) / kWarps, cap = (int64_t)num_sms() * 16;
    return (unsigned)(blocks < cap ? blocks : cap);
}

template <typename T>
void launch_prologue(dsa_dtype fmt, const PrologueArgs &a, cudaStream_t st) {
    const unsigned grid = warp_grid(a.rows);
    if (fmt == DSA_BF16)
        latent_prologue_kernel<DSA_BF16, T><<<grid, 32 * kWarps, 0, st>>>(a);
    else if (fmt == DSA_FP8_LATENT)
        latent_prologue_kernel<DSA_FP8_LATENT, T><<<grid, 32 * kWarps, 0, st>>>(a);
    else
        latent_prologue_kernel<DSA_Q4_LATENT, T><<<grid, 32 * kWarps, 0, st>>>(a);
}

template <typename T>
void launch_read(dsa_dtype fmt, const uint8_t *cache, int64_t t_max, const int32_t *idx, int64_t start_pos,
                 int64_t rows, int64_t n, int dc, int dr, T *out, cudaStream_t st) {
    const unsigned grid = warp_grid(rows);
    int *err = device_error_word();
    if (fmt == DSA_BF16)
        latent_read_kernel<DSA_BF16, T><<<grid, 32 * kWarps, 0, st>>>(cache, t_max, idx, start_pos, rows, n, dc, dr, out, err);
    else if (fmt == DSA_FP8_LATENT)
        latent_read_kernel<DSA_FP8_LATENT, T><<<grid, 32 * kWarps, 0, st>>>(cache, t_max, idx, start_pos, rows, n, dc, dr, out, err);
    else
        latent_read_kernel<DSA_Q4_LATENT, T><<<grid, 32 * kWarps, 0, st>>>(cache, t_max, idx, start_pos, rows, n, dc, dr, out, err);
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
    if (B < 0 || S < 0 || start_pos < 0) return DSA_ERR_INVALID_ARG;
    if (x_dtype != DSA_F32 && x_dtype != DSA_BF16) return DSA_ERR_INVALID_ARG;
    if (cache_dt != DSA_BF16 && cache_dt != DSA_FP8_LATENT && cache_dt != DSA_Q4_LATENT)
        return DSA_ERR_INVALID_ARG;
    if (!dsa::latent_shape_ok(dc, dr)) return DSA_ERR_UNSUPPORTED;
    if (start_pos + S > t_max) return DSA_ERR_INVALID_ARG;
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
        dsa::launch_prologue<__nv_bfloat16>(cache_dt, a, st);
    else
        dsa::launch_prologue<float>(cache_dt, a, st);
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
    if (!idx && start_pos + n > t_max) return DSA_ERR_INVALID_ARG;
    if (B == 0 || n == 0) return DSA_OK;
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
