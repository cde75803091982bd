// latent_attn.cu -- sparse latent attention over a 4-bit cache, and over
// selected blocks of a bf16, FP8 or 4-bit cache.
//
// For each query row (b, s) at position i = start_pos + s and each head, over
// the selected latent rows c_j (key and value, MQA mode):
//   z_j = sm_scale * q . c_j,   out = sum_j softmax(z)_j c_j[:dc],
//   lse = log sum_j exp(z_j)
// A selection is a list of positions, or a list of finished blocks (block e is
// the tokens [e m, e m + m), finished once e < (i + 1) / m) to which the
// query's own unfinished block, the last (i + 1) mod m positions, is added as
// slot 0.
//
// One warp per (query row, head): lane l holds the latent values
// [8 l, 8 l + 8) and [8 l + 256, 8 l + 264) and the rotary pair l of the query
// and of each row, and walks the selection with an online softmax.
#include "latent_rows.cuh"

namespace dsa {
namespace {

constexpr int kHeadsPerCta = 8;

template <int F>
__global__ void __launch_bounds__(32 * kHeadsPerCta)
latent_attn_kernel(const __nv_bfloat16 *__restrict__ q, const uint8_t *__restrict__ kv, int64_t t_max,
                   const int32_t *__restrict__ sel, int n_sel, int block, int S, int Hq, int dc, int dr,
                   int64_t start_pos, float sm_scale, __nv_bfloat16 *__restrict__ out,
                   float *__restrict__ lse, int *err) {
    const int lane = threadIdx.x & 31;
    const int head = blockIdx.y * kHeadsPerCta + (threadIdx.x >> 5);
    const int64_t row = blockIdx.x, b = row / S, s = row - b * S;
    if (head >= Hq) return;
    const int64_t limit = start_pos + s;
    const int64_t rb = latent_fmt_row_bytes(F, dc, dr);
    const int chunks = dc / 8;
    const __nv_bfloat16 *qh = q + (row * Hq + head) * (dc + dr);
    float qv[2][8], o[2][8], q0 = 0.f, q1 = 0.f;
#pragma unroll
    for (int u = 0; u < 2; u++)
#pragma unroll
        for (int e = 0; e < 8; e++) {
            const int d = 8 * (lane + 32 * u) + e;
            qv[u][e] = d < dc ? __bfloat162float(qh[d]) : 0.f;
            o[u][e] = 0.f;
        }
    if (lane < dr / 2) {
        q0 = __bfloat162float(qh[dc + 2 * lane]);
        q1 = __bfloat162float(qh[dc + 2 * lane + 1]);
    }
    float m = -INFINITY, l = 0.f;
    const int32_t *list = sel + row * n_sel;
    // block = 0: the list holds positions
    const int64_t done = block ? (limit + 1) / block : 0;
    const int64_t slots = block ? (int64_t)(n_sel + 1) * block : n_sel;
    for (int64_t j = 0; j < slots; j++) {
        int64_t t;
        if (block) {
            const int64_t e = j / block;
            const int64_t blk = e == 0 ? done : list[e - 1];
            if (blk < 0 || (e > 0 && blk >= done)) continue;
            t = blk * block + (j - e * block);
        } else {
            t = list[j];
        }
        if (t < 0 || t > limit) continue;
        if (t >= t_max) {
            if (lane == 0) record_error(err, DSA_ERR_DEVICE);
            continue;
        }
        const uint8_t *c = kv + (b * t_max + t) * rb;
        float cv[2][8], part = 0.f;
#pragma unroll
        for (int u = 0; u < 2; u++) {
            const uint4 w = lane + 32 * u < chunks ? latent_chunk8<F>(c, dc, dr, lane + 32 * u)
                                                   : make_uint4(0, 0, 0, 0);
            const uint32_t ws[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
            for (int e = 0; e < 4; e++) {
                const float2 f = bf16x2_to_f32(ws[e]);
                cv[u][2 * e] = f.x;
                cv[u][2 * e + 1] = f.y;
            }
#pragma unroll
            for (int e = 0; e < 8; e++) part = fmaf(qv[u][e], cv[u][e], part);
        }
        if (lane < dr / 2) {
            const float2 f = bf16x2_to_f32(reinterpret_cast<const uint32_t *>(c + latent_rope_at<F>(dc))[lane]);
            part = fmaf(q0, f.x, fmaf(q1, f.y, part));
        }
        const float z = warp_sum(part) * sm_scale;
        if (z == -INFINITY) continue;              // weight 0 (and no reference to subtract)
        const float m_new = fmaxf(m, z);
        const float corr = m == m_new ? 1.f : expf(m - m_new);
        const float p = expf(z - m_new);
        l = fmaf(l, corr, p);
#pragma unroll
        for (int u = 0; u < 2; u++)
#pragma unroll
            for (int e = 0; e < 8; e++) o[u][e] = fmaf(o[u][e], corr, p * cv[u][e]);
        m = m_new;
    }
    const float inv = l > 0.f ? 1.f / l : (l == 0.f ? 0.f : l);
    __nv_bfloat16 *oh = out + (row * Hq + head) * dc;
#pragma unroll
    for (int u = 0; u < 2; u++) {
        if (lane + 32 * u >= chunks) continue;
        uint32_t w[4];
#pragma unroll
        for (int e = 0; e < 4; e++) w[e] = bf16x2_bits(__floats2bfloat162_rn(o[u][2 * e] * inv, o[u][2 * e + 1] * inv));
        reinterpret_cast<uint4 *>(oh)[lane + 32 * u] = make_uint4(w[0], w[1], w[2], w[3]);
    }
    if (lse && lane == 0) lse[row * Hq + head] = l == 0.f ? -INFINITY : m + logf(l);
}

}  // namespace

size_t latent_attn_workspace_bytes(int B, int S, int Hq, int dc, int dr, int n_sel, int block) { return 0; }

dsa_status launch_latent_attn(const void *q, const void *kv, dsa_dtype fmt, int64_t t_max, const int32_t *sel,
                              int n_sel, int block, int B, int S, int Hq, int dc, int dr, int64_t start_pos,
                              float sm_scale, void *out, float *lse, void *ws, cudaStream_t st) {
    const dim3 grid((unsigned)((int64_t)B * S), (unsigned)((Hq + kHeadsPerCta - 1) / kHeadsPerCta));
    int *err = device_error_word();
    auto run = [&](auto kernel) {
        kernel<<<grid, 32 * kHeadsPerCta, 0, st>>>(
            static_cast<const __nv_bfloat16 *>(q), static_cast<const uint8_t *>(kv), t_max, sel, n_sel, block, S,
            Hq, dc, dr, start_pos, sm_scale, static_cast<__nv_bfloat16 *>(out), lse, err);
    };
    if (fmt == DSA_BF16)
        run(latent_attn_kernel<DSA_BF16>);
    else if (fmt == DSA_FP8_LATENT)
        run(latent_attn_kernel<DSA_FP8_LATENT>);
    else
        run(latent_attn_kernel<DSA_Q4_LATENT>);
    return launch_status();
}

namespace {

// The checks that both entry points share.  DSA_OK with *run = false: nothing to do.
dsa_status check_attn(const void *q, const void *kv, int64_t t_max, const int32_t *sel, int n_sel, int block,
                      int B, int S, int Hq, int dc, int dr, int64_t start_pos, const void *out, const float *lse,
                      const void *ws, size_t ws_bytes, bool *run) {
    *run = false;
    if (B < 0 || S < 0 || Hq < 0 || n_sel < 1 || start_pos < 0) return DSA_ERR_INVALID_ARG;
    if (!latent_shape_ok(dc, dr)) return DSA_ERR_UNSUPPORTED;
    if (Hq > 1024 || block > 1 << 20) return DSA_ERR_UNSUPPORTED;
    if ((int64_t)B * S * Hq == 0) return DSA_OK;
    if (start_pos + S > t_max || t_max > INT32_MAX) return DSA_ERR_INVALID_ARG;
    if ((int64_t)B * S * n_sel > INT32_MAX || (int64_t)B * S * Hq > INT32_MAX ||
        (int64_t)(n_sel + 1) * (block ? block : 1) > INT32_MAX)
        return DSA_ERR_UNSUPPORTED;
    if (!q || !kv || !sel || !out) return DSA_ERR_INVALID_ARG;
    if (!aligned16(q) || !aligned16(kv) || !aligned16(out) || (reinterpret_cast<uintptr_t>(sel) & 3) ||
        (reinterpret_cast<uintptr_t>(lse) & 3))
        return DSA_ERR_INVALID_ARG;
    const size_t need = latent_attn_workspace_bytes(B, S, Hq, dc, dr, n_sel, block);
    if (need > 0 && (!ws || ws_bytes < need || !aligned16(ws))) return DSA_ERR_WORKSPACE;
    *run = true;
    return DSA_OK;
}

}  // namespace
}  // namespace dsa

extern "C" size_t dsa_sparse_mla_attn_q4_workspace_size(int B, int S, int Hq, int dc, int dr, int k) {
    if (B <= 0 || S <= 0 || Hq <= 0 || k <= 0 || !dsa::latent_shape_ok(dc, dr)) return 0;
    return dsa::latent_attn_workspace_bytes(B, S, Hq, dc, dr, k, 0);
}

extern "C" dsa_status dsa_sparse_mla_attn_q4(const void *q, const uint8_t *kv_q4, int64_t t_max,
                                             const int32_t *idx, int B, int S, int Hq, int dc, int dr,
                                             int k, int64_t start_pos, float sm_scale, void *out,
                                             float *lse, void *workspace, size_t workspace_bytes,
                                             dsa_stream_t stream) {
    bool run = false;
    const dsa_status st = dsa::check_attn(q, kv_q4, t_max, idx, k, 0, B, S, Hq, dc, dr, start_pos, out, lse,
                                          workspace, workspace_bytes, &run);
    if (st != DSA_OK || !run) return st;
    return dsa::launch_latent_attn(q, kv_q4, DSA_Q4_LATENT, t_max, idx, k, 0, B, S, Hq, dc, dr, start_pos,
                                   sm_scale, out, lse, workspace, reinterpret_cast<cudaStream_t>(stream));
}

extern "C" size_t dsa_block_mla_attn_workspace_size(int B, int S, int Hq, int dc, int dr, int kb, int block) {
    if (B <= 0 || S <= 0 || Hq <= 0 || kb <= 0 || block <= 0 || !dsa::latent_shape_ok(dc, dr)) return 0;
    return dsa::latent_attn_workspace_bytes(B, S, Hq, dc, dr, kb, block);
}

extern "C" dsa_status dsa_block_mla_attn(const void *q, const void *kv_cache, dsa_dtype cache_dt,
                                         int64_t t_max, const int32_t *blk, int B, int S, int Hq,
                                         int dc, int dr, int kb, int block, int64_t start_pos,
                                         float sm_scale, void *out, float *lse, void *workspace,
                                         size_t workspace_bytes, dsa_stream_t stream) {
    if (cache_dt != DSA_BF16 && cache_dt != DSA_FP8_LATENT && cache_dt != DSA_Q4_LATENT)
        return DSA_ERR_INVALID_ARG;
    if (block < 1) return DSA_ERR_INVALID_ARG;
    bool run = false;
    const dsa_status st = dsa::check_attn(q, kv_cache, t_max, blk, kb, block, B, S, Hq, dc, dr, start_pos, out,
                                          lse, workspace, workspace_bytes, &run);
    if (st != DSA_OK || !run) return st;
    return dsa::launch_latent_attn(q, kv_cache, cache_dt, t_max, blk, kb, block, B, S, Hq, dc, dr, start_pos,
                                   sm_scale, out, lse, workspace, reinterpret_cast<cudaStream_t>(stream));
}
