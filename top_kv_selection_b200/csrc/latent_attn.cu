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
// Tensor-core form, transposed: the keys are the MMA's M, the heads its N.
//   S^T[key, head] = C Q^T       M = 128 slots, N = 16, 32 or 64 heads, K = dc + dr
//   O^T[dc, head] += C^T P^T     M = 128 columns of dc at a time, K = 128 slots
// so the output of a CTA's heads takes dc / 128 x N TMEM columns (256 for 64
// heads of 512 columns) and the logits have room beside it: one CTA walks any
// number of 128-slot tiles of its query row with an online softmax, without
// leaving TMEM, and few heads cost few columns.  (With the heads as M, 512
// output columns fill TMEM and each tile's result has to leave it.)
//
// One CTA = (query row, group of up to 64 heads, share of the row's slots).  (One
// that stays and takes row after row, the output written under the next row's
// logits, needs more registers than there are for 4-bit rows, 1012 against 948 us
// at 1024 queries, and gains nothing for bf16 ones.)
//
// Sixteen work warps and one that issues the MMAs.  Per tile, a work warp
//   - decodes the tile's rows (eight threads a row, two rows a thread) to bf16
//     in 64-column chunks, 128B-swizzled K-major tiles that serve as the logits'
//     A operand and, read MN-major, as the value mix's, as the value mix of the
//     tile before frees each pair of chunks.  Quantised rows wait in registers
//     since one tile ahead; bf16 rows are copied by cp.async, their lines
//     requested into L2 one tile ahead.  The weights P take the place of the
//     rotary chunk, which the logits have read by then;
//   - loads the next tile's rows;
//   - takes the softmax of (slot, quarter of the heads): the running maximum of
//     each head is a reference kept until a logit passes it by more than 8 (2^8
//     in the weights, which bf16 and the fp32 sums hold at full precision);
//     only then are the tile's maxima reduced and the output rescaled.  Sums
//     stay per thread in fp32 and are reduced once at the end; the weights are
//     rounded to bf16 as MMA operands (the sums take them unrounded).
// Shared memory bounds the walk: a 128 x 64 x 16 MMA reads 6 KB in its 49
// cycles, and the decoded tile is written beside it: 570 KB a tile, 2.3 of the
// 3.8 us that one takes.  1024 queries of 2048 slots and 128 heads take 945 us
// (618 TFLOP/s) over 4-bit rows, 8 queries 20.5 us.
// Splits of a row (when there are fewer rows than SMs) leave fp32 partials that
// a second kernel merges (fp16 ones with a power of two per 32 columns halved
// the bytes, but the maxima they need cost more than the bytes: 24.9 against
// 21.2 us at eight rows of 2048 slots).
#include <cfloat>
#include <cmath>

#include "latent_rows.cuh"
#include "tc_ptx.cuh"

namespace dsa {
namespace {

constexpr int kTile = 128;                      // slots per tile (the MMA M of the logits)
constexpr int kRegion = kTile * 128;            // one 64-column chunk of a tile: 16 KB
constexpr int kWork = 512;                      // work threads
constexpr int kThreads = kWork + 32;
constexpr int kMaxHeads = 64;                   // heads per CTA
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
// stands for a head's reference until it has one: the lowest number, so that every
// finite logit above it passes it by more than the slack (kLeastScale times 2^128 is
// 32); -inf - kUnseen is -inf
constexpr float kUnseen = -FLT_MAX;
constexpr float kLeastScale = 0x1p-123f;
constexpr float kSlack = 8.f;                   // how far (log2) a logit may pass the reference

struct AttnArgs {
    const __nv_bfloat16 *q;     // [rows, Hq, dc + dr]
    const uint8_t *kv;          // [B, t_max, row]
    const int32_t *sel;         // [rows, n_sel] positions or block ids
    __nv_bfloat16 *out;
    float *lse;
    float *part_o;              // [units][heads][dc] (splits > 1)
    float2 *part_ml;            // [units][heads] (reference, sum)
    int64_t t_max, start_pos, row_bytes;
    int n_sel, block, slots;    // block = 0: the list holds positions
    int S, Hq, dc, dr;
    int groups, splits, split_slots;
    float scale;                // |sm_scale| * log2(e), at least kLeastScale
    float sign;                 // of sm_scale
    int *err;
};

// Control block behind the tiles and the query.
struct alignas(16) Control {
    float red[4][kMaxHeads];    // per TMEM lane quarter: maxima, later sums
    float ref[kMaxHeads];       // the heads' references, of sign * q . c (-inf: no logit seen)
    float sub[kMaxHeads];       // what is subtracted: the reference, or kUnseen
    float fac[kMaxHeads];       // rescaling of this tile; at the end 1 / sum
    uint64_t full[5];           // chunk pair m (4: the rotary chunk) is in shared memory
    uint64_t q_full, s_done, p_full, mma_fin;
    uint64_t o_done[4];         // value mix of dc columns [128 m, 128 m + 128) is complete
    uint32_t tmem;
    int abort;
    int last;                   // last slot of the share that counts
    uint8_t valid[2][kTile / 4];   // per tile parity: four slots a byte, a bit for each that counts
};

size_t smem_bytes(int dc, int nh) {
    return 1024 + (size_t)(dc / 64 + 1) * (kRegion + nh * 128) + sizeof(Control);
}

__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src, uint32_t src_bytes) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(src_bytes) : "memory");
}
// Arrives on `bar` once every cp.async this thread issued so far has landed.
__device__ __forceinline__ void cp_async_arrive(uint64_t *bar) {
    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(tc::smem_u32(bar)) : "memory");
}
__device__ __forceinline__ void st_shared_v4(uint32_t addr, uint4 v) {
    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w)
                 : "memory");
}
// Loads that stay behind griddepcontrol.wait (volatile, coherent).
__device__ __forceinline__ uint4 ld_v4(const void *p) {
    uint4 v;
    asm volatile("ld.global.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
    return v;
}
__device__ __forceinline__ uint2 ld_v2(const void *p) {
    uint2 v;
    asm volatile("ld.global.v2.b32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "l"(p));
    return v;
}
__device__ __forceinline__ uint32_t ld_b32(const void *p) {
    uint32_t v;
    asm volatile("ld.global.b32 %0, [%1];" : "=r"(v) : "l"(p));
    return v;
}
// 16 bytes that are 16-byte aligned (wide) or 4-byte aligned
__device__ __forceinline__ uint4 ld_piece(const uint8_t *p, bool wide) {
    if (wide) return ld_v4(p);
    return make_uint4(ld_b32(p), ld_b32(p + 4), ld_b32(p + 8), ld_b32(p + 12));
}
// 2^x by the SFU (relative error about 2^-22; 2^-inf = +0).
__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// a softmax thread's columns
__device__ __forceinline__ void ld_cols(uint32_t taddr, uint32_t (&v)[8]) { tc::tmem_ld8(taddr, v); }
__device__ __forceinline__ void ld_cols(uint32_t taddr, uint32_t (&v)[16]) { tc::tmem_ld16(taddr, v); }
// Reduces N values over the warp's lanes: lanes trade halves of their values
// until each holds one, or a part of one, in v[0]; returns which one that is
// (the lanes that differ in the bits below 32 / N only hold the same).  N
// shuffles; a redux for each value measured slower.
template <int N, typename Op>
__device__ __forceinline__ int reduce_lanes(float (&v)[N], Op op) {
    const int lane = threadIdx.x & 31;
    int which = 0;
#pragma unroll
    for (int m = 16, n = N / 2; m > 0; m >>= 1, n >>= 1) {
        const bool up = lane & m;
        if (n > 0) {
            which += up ? n : 0;
#pragma unroll
            for (int e = 0; e < n; e++) {
                const float give = up ? v[e] : v[e + n], keep = up ? v[e + n] : v[e];
                v[e] = op(keep, __shfl_xor_sync(0xffffffffu, give, m));
            }
        } else {
            v[0] = op(v[0], __shfl_xor_sync(0xffffffffu, v[0], m));
        }
    }
    return which;
}

// The cache row of a selection slot of query row `row`, or -1.  Slot 0's block
// is the query's unfinished one; `limit` < t_max, so every position that is
// not ahead of the query lies in the cache.
__device__ __forceinline__ int32_t slot_row(const AttnArgs &a, const int32_t *list, int slot, int limit, int done) {
    if (slot >= a.slots) return -1;
    int32_t t;
    if (a.block == 0) {
        t = (int32_t)ld_b32(list + slot);
    } else {
        const int e = (int)((unsigned)slot / (unsigned)a.block);
        const int32_t b = e == 0 ? done : (int32_t)ld_b32(list + e - 1);
        if (b < 0 || (e > 0 && b >= done)) return -1;
        const int64_t p = (int64_t)b * a.block + (slot - e * a.block);
        t = p > limit ? -1 : (int32_t)p;
    }
    return t < 0 || t > limit ? -1 : t;
}

// What a thread holds of the next tile: eight threads p share two rows.  Of
// 4-bit codes a thread takes a group of its own row (row 0 for p < 4, else row
// 1) in each chunk pair; of wider ones 16 bytes of every 128 of both rows.
template <int F> struct RawRows;
template <> struct RawRows<DSA_Q4_LATENT> {
    uint4 code[4];              // groups 4 m + h, h = p & 3
    uint2 scale;                // of groups 4 h .. 4 h + 3
    uint4 rope0, rope1;
};
template <> struct RawRows<DSA_FP8_LATENT> {
    uint4 x0[4], x1[4];         // codes [16 p, 16 p + 16) of block m
    float s0, s1;               // block p & 3
    uint4 rope0, rope1;
};
template <> struct RawRows<DSA_BF16> {
    uint4 rope0, rope1;
};

template <int F>
__device__ __forceinline__ void load_rows(RawRows<F> &r, const AttnArgs &a, int64_t rbase, int32_t t0, int32_t t1,
                                          int p) {
    const uint8_t *row0 = a.kv + (rbase + (t0 < 0 ? 0 : t0)) * a.row_bytes;
    const uint8_t *row1 = a.kv + (rbase + (t1 < 0 ? 0 : t1)) * a.row_bytes;
    const bool v0 = t0 >= 0, v1 = t1 >= 0;
    // (FP8 rows of other widths than 512 are only 4-byte aligned)
    const bool wide = F != DSA_FP8_LATENT || (a.row_bytes & 15) == 0;
    const uint4 zero = make_uint4(0, 0, 0, 0);
    if constexpr (F == DSA_Q4_LATENT) {
        const int h = p & 3;
        const uint8_t *row = p < 4 ? row0 : row1;
        const bool v = p < 4 ? v0 : v1;
#pragma unroll
        for (int m = 0; m < 4; m++) r.code[m] = v && 128 * m < a.dc ? ld_v4(row + 64 * m + 16 * h) : zero;
        r.scale = v && 128 * h < a.dc ? ld_v2(row + latent_q4_scales_at(a.dc, a.dr) + 8 * h) : make_uint2(0, 0);
    } else if constexpr (F == DSA_FP8_LATENT) {
#pragma unroll
        for (int m = 0; m < 4; m++) {
            r.x0[m] = v0 && 128 * m < a.dc ? ld_piece(row0 + 128 * m + 16 * p, wide) : zero;
            r.x1[m] = v1 && 128 * m < a.dc ? ld_piece(row1 + 128 * m + 16 * p, wide) : zero;
        }
        const bool on = 128 * (p & 3) < a.dc;
        r.s0 = v0 && on ? __uint_as_float(ld_b32(row0 + a.dc + 4 * (p & 3))) : 0.f;
        r.s1 = v1 && on ? __uint_as_float(ld_b32(row1 + a.dc + 4 * (p & 3))) : 0.f;
    } else if (p == 0) {
        if (v0) tc::prefetch_l2_bulk(row0, (uint32_t)a.row_bytes);
        if (v1) tc::prefetch_l2_bulk(row1, (uint32_t)a.row_bytes);
    }
    const int at = latent_rope_at<F>(a.dc) + 16 * p;
    r.rope0 = v0 && 8 * p < a.dr ? ld_piece(row0 + at, wide) : zero;
    r.rope1 = v1 && 8 * p < a.dr ? ld_piece(row1 + at, wide) : zero;
}

// Decodes the thread's share of chunk pair m into the tile (rows j0, j1).  The
// order in which a thread stores its 16-byte units is turned by its chunk, so
// that with the swizzle eight threads that store together touch all banks once
// (j1 differs from j0 in the lowest bit).
template <int F>
__device__ __forceinline__ void store_pair(const RawRows<F> &r, int m, uint32_t tile, int p, int j0, int j1) {
    if constexpr (F == DSA_Q4_LATENT) {
        // group 4 m + h: chunk 2 m + (h >> 1), units 4 (h & 1) + 0..3
        const int h = p & 3, up = h >> 1, j = p < 4 ? j0 : j1, sw = j & 7;
        const uint32_t x = __shfl_sync(0xffffffffu, r.scale.x, m, 4), y = __shfl_sync(0xffffffffu, r.scale.y, m, 4);
        const uint32_t two = up ? y : x;
        const __nv_bfloat16 s1 = __ushort_as_bfloat16((uint16_t)((h & 1) ? two >> 16 : two));
        const __nv_bfloat162 s = __halves2bfloat162(s1, s1);
        const uint4 c = r.code[m];
        const uint32_t w[4] = {up ? c.z : c.x, up ? c.w : c.y, up ? c.x : c.z, up ? c.y : c.w};
        const uint32_t dst = tile + (2 * m + up) * kRegion + j * 128;
#pragma unroll
        for (int u = 0; u < 4; u++)
            st_shared_v4(dst + (((4 * (h & 1) + (u ^ (2 * up))) ^ sw) << 4), q4_decode8(w[u], s));
    } else if constexpr (F == DSA_FP8_LATENT) {
        // codes [16 p, 16 p + 16) of block m: chunk 2 m + (p >> 2), units 2 (p & 3) + 0, 1
        const int up = p >> 2, u0 = 2 * (p & 3);
        const float c0 = __shfl_sync(0xffffffffu, r.s0, m, 8), c1 = __shfl_sync(0xffffffffu, r.s1, m, 8);
        const uint32_t dst = tile + (2 * m + up) * kRegion;
        const uint4 a = r.x0[m], b = r.x1[m];
        const int w0 = (u0 + up) ^ (j0 & 7), w1 = (u0 + up) ^ (j1 & 7);
        st_shared_v4(dst + j0 * 128 + (w0 << 4), fp8_decode8(up ? a.z : a.x, up ? a.w : a.y, c0));
        st_shared_v4(dst + j0 * 128 + ((w0 ^ 1) << 4), fp8_decode8(up ? a.x : a.z, up ? a.y : a.w, c0));
        st_shared_v4(dst + j1 * 128 + (w1 << 4), fp8_decode8(up ? b.z : b.x, up ? b.w : b.y, c1));
        st_shared_v4(dst + j1 * 128 + ((w1 ^ 1) << 4), fp8_decode8(up ? b.x : b.z, up ? b.y : b.w, c1));
    }
}

template <int F, int NH>
__global__ void __launch_bounds__(kThreads, 1) latent_attn_kernel(const AttnArgs a) {
    // heads per work thread (of 16 heads, the first two quarters take eight each)
    constexpr int kCols = NH == 16 ? 8 : NH / 4;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *sm = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const int nc = a.dc / 64, mt = a.dc / 128;             // latent chunks, dc tiles
    uint8_t *qs = sm + (nc + 1) * kRegion;
    Control &ctl = *reinterpret_cast<Control *>(qs + (nc + 1) * NH * 128);
    volatile int *abort = &ctl.abort;
    const uint32_t tile = tc::smem_u32(sm), qbase = tc::smem_u32(qs);
    const uint32_t pbase = tile + nc * kRegion;            // P takes the rotary chunk's place
    // (read through a shuffle, so that it is known to be the same in a warp)
    const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;

    // TMEM: the logits, then the output tiles
    const uint32_t ncols = NH * (mt + 1) <= 32 ? 32 : NH * (mt + 1) <= 64 ? 64 : NH * (mt + 1) <= 128 ? 128
                           : NH * (mt + 1) <= 256 ? 256 : 512;
    if (warp == kWork / 32) {
        if (lane == 0) {
            // (a warp arrives once; copies in flight arrive for each thread)
            for (int i = 0; i < 4; i++) tc::mbar_init(&ctl.full[i], F == DSA_BF16 ? kWork : kWork / 32);
            tc::mbar_init(&ctl.full[4], kWork / 32);
            tc::mbar_init(&ctl.q_full, kWork);
            tc::mbar_init(&ctl.s_done, 1);
            tc::mbar_init(&ctl.p_full, 1);
            tc::mbar_init(&ctl.mma_fin, 1);
            for (int i = 0; i < 4; i++) tc::mbar_init(&ctl.o_done[i], 1);
            ctl.abort = 0;
            ctl.last = -1;
            tc::fence_mbar_init();
        }
        __syncwarp();
        tc::tmem_alloc(&ctl.tmem, ncols);
        tc::tmem_relinquish();
    }
    if (threadIdx.x < NH) {
        ctl.ref[threadIdx.x] = -INFINITY;
        ctl.sub[threadIdx.x] = kUnseen;
    }
    tc::tc_fence_before();
    __syncthreads();
    tc::tc_fence_after();
    const uint32_t tmem = __shfl_sync(0xffffffffu, ctl.tmem, 0);
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    // every global read comes after this (a no-op without a programmatic launch)
    asm volatile("griddepcontrol.wait;" ::: "memory");

    // blockIdx.x = (row * groups + g) * splits + sp
    const int sp = (int)(blockIdx.x % (unsigned)a.splits);
    const unsigned rg = blockIdx.x / (unsigned)a.splits;
    const int g = (int)(rg % (unsigned)a.groups);
    const int64_t row = rg / (unsigned)a.groups;
    const int64_t b = row / a.S;
    const int limit = (int)(a.start_pos + (row - b * a.S));
    const int done = a.block ? (limit + 1) / a.block : 0;
    const int32_t *list = a.sel + row * a.n_sel;
    const int lo = sp * a.split_slots;
    const int hi = lo + a.split_slots < a.slots ? lo + a.split_slots : a.slots;
    const int h0 = g * kMaxHeads;                          // first head
    const int heads = a.Hq - h0 < NH ? a.Hq - h0 : NH;
    const int64_t rbase = b * a.t_max;

    // The walk goes as far as the share's last slot that counts, and over one
    // tile at least (a share of one tile is not looked through).
    const bool one_tile = hi - lo <= kTile;
    bool ok = true;
    int tiles = 1;

    if (warp < kWork / 32) {
        const int t = threadIdx.x;
        // gather: two rows of the tile, 16 bytes of each 128
        const int p8 = t & 7, j0 = t >> 3, j1 = kTile / 2 + (j0 ^ 1);
        const int q4 = warp & 3, c = warp >> 2;            // softmax: TMEM lane quarter, quarter of the heads
        const bool active = c * kCols < NH;
        const int key = q4 * 32 + lane;
        const uint32_t lane_addr = (uint32_t)(q4 * 32) << 16;
        const int dqk = a.dc + a.dr;
        auto row_of = [&](int i, int j) {                  // the cache row of tile i's row j
            const int s = lo + i * kTile + j;
            return slot_row(a, list, s < hi ? s : a.slots, limit, done);
        };
        const int own = p8 < 4 ? j0 : j1;
        int32_t town = row_of(0, own);
        // the query, as nc + 1 K-major blocks of 64 columns (absent heads and
        // columns are zero-filled)
        const __nv_bfloat16 *q = a.q + (row * a.Hq + h0) * dqk;
        for (int f = t; f < (nc + 1) * NH * 8; f += kWork) {
            const int p = f & 7, head = (f >> 3) % NH, blk = (f >> 3) / NH;
            const bool v = head < heads && blk * 64 + p * 8 < dqk;
            cp_async16(qbase + blk * NH * 128 + head * 128 + ((p ^ (head & 7)) << 4),
                       q + (v ? head * dqk + blk * 64 + p * 8 : 0), v ? 16u : 0u);
        }
        cp_async_arrive(&ctl.q_full);
        RawRows<F> raw;
        int32_t t0 = __shfl_sync(0xffffffffu, town, 0, 8), t1 = __shfl_sync(0xffffffffu, town, 4, 8);
        // which of a tile's slots count, by one bit each, for the softmax: known
        // a tile ahead, so that the barriers between order it
        auto note_valid = [&](int i) {
            // the warp's rows 4 warp .. 4 warp + 3 and those 64 further on
            // (which trade places in pairs)
            const uint32_t x0 = __ballot_sync(0xffffffffu, t0 >= 0), x1 = __ballot_sync(0xffffffffu, t1 >= 0);
            auto pack = [](uint32_t x) { return (x & 1) | (x >> 7 & 2) | (x >> 14 & 4) | (x >> 21 & 8); };
            if (lane == 0) {
                const uint32_t y = pack(x1);
                ctl.valid[i & 1][warp] = (uint8_t)pack(x0);
                ctl.valid[i & 1][kTile / 8 + warp] = (uint8_t)((y & 5) << 1 | (y >> 1 & 5));
            }
        };
        note_valid(0);
        load_rows<F>(raw, a, rbase, t0, t1, p8);
        tc::named_barrier(1, kWork);
        town = row_of(1, own);
        float lsum[kCols];
#pragma unroll
        for (int e = 0; e < kCols; e++) lsum[e] = 0.f;
        const uint32_t scol = tmem + lane_addr + c * kCols;
        for (int i = 0; i < tiles; i++) {
            // chunk pair m is free once the value mix m of the tile before is
            // complete; the rotary chunk (and P) once all of it is
#pragma unroll
            for (int m = 0; m < 4; m++) {
                if (m >= mt) break;
                if (i > 0 && !tc::mbar_wait(&ctl.o_done[m], (i - 1) & 1, a.err, abort)) ok = false;
                if constexpr (F == DSA_BF16) {
                    const int64_t r0 = (rbase + (t0 < 0 ? 0 : t0)) * a.row_bytes + 256 * m + 16 * p8;
                    const int64_t r1 = (rbase + (t1 < 0 ? 0 : t1)) * a.row_bytes + 256 * m + 16 * p8;
                    const uint32_t d0 = tile + 2 * m * kRegion + j0 * 128 + ((p8 ^ (j0 & 7)) << 4);
                    const uint32_t d1 = tile + 2 * m * kRegion + j1 * 128 + ((p8 ^ (j1 & 7)) << 4);
                    cp_async16(d0, a.kv + r0, t0 < 0 ? 0u : 16u);
                    cp_async16(d1, a.kv + r1, t1 < 0 ? 0u : 16u);
                    cp_async16(d0 + kRegion, a.kv + r0 + 128, t0 < 0 ? 0u : 16u);
                    cp_async16(d1 + kRegion, a.kv + r1 + 128, t1 < 0 ? 0u : 16u);
                    cp_async_arrive(&ctl.full[m]);
                } else {
                    store_pair<F>(raw, m, tile, p8, j0, j1);
                    __syncwarp();
                    if (lane == 0) tc::mbar_arrive(&ctl.full[m]);
                }
            }
            st_shared_v4(pbase + j0 * 128 + ((p8 ^ (j0 & 7)) << 4), raw.rope0);
            st_shared_v4(pbase + j1 * 128 + ((p8 ^ (j1 & 7)) << 4), raw.rope1);
            __syncwarp();
            if (lane == 0) tc::mbar_arrive(&ctl.full[4]);
            t0 = __shfl_sync(0xffffffffu, town, 0, 8);
            t1 = __shfl_sync(0xffffffffu, town, 4, 8);
            note_valid(i + 1);
            load_rows<F>(raw, a, rbase, t0, t1, p8);       // (rows past the share's end are -1)
            town = row_of(i + 2, own);
            if (i == 0 && !one_tile) {
                int mine = -1;
#pragma unroll 4
                for (int s = lo + t; s < hi; s += kWork)
                    if (slot_row(a, list, s, limit, done) >= 0) mine = s;
                mine = __reduce_max_sync(0xffffffffu, mine);
                if (lane == 0 && mine >= 0) atomicMax(&ctl.last, mine);
                tc::named_barrier(2, kThreads);
                const int last = __shfl_sync(0xffffffffu, ctl.last, 0);
                tiles = last < lo ? 1 : (last - lo) / kTile + 1;
            }
            if (!tc::mbar_wait(&ctl.s_done, i & 1, a.err, abort)) ok = false;
            tc::tc_fence_after();
            const bool valid = ctl.valid[i & 1][key >> 2] >> (key & 3) & 1;
            // weights against the standing references; whether a logit passes
            // its reference by too much is known to all only behind them
            float p[kCols];
            bool over = false;
            auto weights = [&]() {
                uint32_t v[kCols];
                ld_cols(scol, v);
                tc::tmem_wait_ld();
#pragma unroll
                for (int x = 0; x < kCols; x += 8) {
                    const float4 s0 = *reinterpret_cast<const float4 *>(&ctl.sub[c * kCols + x]);
                    const float4 s1 = *reinterpret_cast<const float4 *>(&ctl.sub[c * kCols + x + 4]);
                    const float sub[8] = {s0.x, s0.y, s0.z, s0.w, s1.x, s1.y, s1.z, s1.w};
                    uint32_t pk[4];
#pragma unroll
                    for (int e = 0; e < 8; e++) {
                        // (the difference before the scale: it is 0 at the maximum
                        // however far that is from zero)
                        const float z = fmaf(__uint_as_float(v[x + e]), a.sign, -sub[e]) * a.scale;
                        over |= z > kSlack;
                        p[x + e] = valid ? ex2(z) : 0.f;
                    }
#pragma unroll
                    for (int e = 0; e < 4; e++) pk[e] = bf16x2_bits(__floats2bfloat162_rn(p[x + 2 * e], p[x + 2 * e + 1]));
                    st_shared_v4(pbase + key * 128 + (((c * (kCols / 8) + x / 8) ^ (key & 7)) << 4),
                                 make_uint4(pk[0], pk[1], pk[2], pk[3]));
                }
            };
            // (no reference stands before the first tile)
            if (i > 0 && active) weights();
            tc::tc_fence_before();
            if (i == 0 || tc::named_barrier_any(1, kWork, over && valid)) {
                // new references: the tile's maxima, per lane quarter and then
                // over the four
                if (active) {
                    uint32_t v[kCols];
                    ld_cols(scol, v);
                    tc::tmem_wait_ld();
#pragma unroll
                    for (int e = 0; e < kCols; e++) p[e] = valid ? __uint_as_float(v[e]) * a.sign : -INFINITY;
                    const int e = reduce_lanes(p, [](float x, float y) { return fmaxf(x, y); });
                    if ((lane & (32 / kCols - 1)) == 0) ctl.red[q4][c * kCols + e] = p[0];
                }
                tc::named_barrier(1, kWork);
                if (t < NH) {
                    const float old = ctl.ref[t];
                    const float m = fmaxf(fmaxf(fmaxf(ctl.red[0][t], ctl.red[1][t]),
                                                fmaxf(ctl.red[2][t], ctl.red[3][t])), old);
                    ctl.fac[t] = old == m ? 1.f : ex2((old - m) * a.scale);
                    ctl.ref[t] = m;
                    ctl.sub[t] = m == -INFINITY ? kUnseen : m;
                }
                tc::named_barrier(1, kWork);
                if (active) {
                    if (i > 0) {
                        // (the value mix of the tile before is complete: this
                        // tile's logits were issued after it)
#pragma unroll
                        for (int e = 0; e < kCols; e++) lsum[e] *= ctl.fac[c * kCols + e];
#pragma unroll 1
                        for (int m = 0; m < mt; m++) {
#pragma unroll 1
                            for (int x = 0; x < kCols; x += 8) {
                                const uint32_t col = scol + NH * (m + 1) + x;
                                uint32_t v[8];
                                tc::tmem_ld8(col, v);
                                tc::tmem_wait_ld();
#pragma unroll
                                for (int e = 0; e < 8; e++)
                                    v[e] = __float_as_uint(__uint_as_float(v[e]) * ctl.fac[c * kCols + x + e]);
                                tc::tmem_st8(col, v);
                            }
                        }
                        tc::tmem_wait_st();
                    }
                    weights();
                }
                tc::tc_fence_before();
                tc::named_barrier(1, kWork);
            }
            // every warp's weights are behind the barrier
            if (t == 0) tc::mbar_arrive(&ctl.p_full);
            if (active) {
#pragma unroll
                for (int e = 0; e < kCols; e++) lsum[e] += p[e];
            }
        }
        // the heads' sums, over the warp's slots and then over the lane quarters
        if (active) {
            const int e = reduce_lanes(lsum, [](float x, float y) { return x + y; });
            if ((lane & (32 / kCols - 1)) == 0) ctl.red[q4][c * kCols + e] = lsum[0];
        }
        tc::named_barrier(1, kWork);
        if (t < heads) {
            const float l = (ctl.red[0][t] + ctl.red[1][t]) + (ctl.red[2][t] + ctl.red[3][t]);
            // (l is NaN where a logit is: it passes through)
            ctl.fac[t] = l == 0.f ? 0.f : 1.f / l;
            if (a.splits > 1)
                // (a NaN sum makes the reference NaN, so that the merge keeps it)
                a.part_ml[(int64_t)blockIdx.x * NH + t] = make_float2(l == 0.f ? -INFINITY : l != l ? l : ctl.ref[t], l);
            else if (a.lse)
                a.lse[row * a.Hq + h0 + t] = l == 0.f ? -INFINITY : fmaf(ctl.ref[t], a.scale, log2f(l)) * kLn2;
        }
    } else {
        // ------------------------------------------------------------- MMA
        {
            // (the whole warp walks, one elected lane issues: uniform control
            // keeps the descriptors in uniform registers)
            const uint32_t id_qk = tc::instr_desc(tc::kFmtBF16, tc::kFmtBF16, 128, NH);
            const uint32_t id_pv = tc::instr_desc(tc::kFmtBF16, tc::kFmtBF16, 128, NH, true, true);
            // (descriptors count 16-byte units: one add per MMA, so that the
            // issue keeps ahead of the tensor core)
            const uint64_t kd0 = tc::smem_desc(tile, 1024, tc::kSwizzle128B);
            const uint64_t qd0 = tc::smem_desc(qbase, 1024, tc::kSwizzle128B);
            const uint64_t vd0 = tc::smem_desc(tile, 1024, tc::kSwizzle128B, kRegion);
            const uint64_t pd0 = tc::smem_desc(pbase, 1024, tc::kSwizzle128B, kRegion);
            const int rope_steps = (a.dr + 15) / 16;
            // (a wait that gave up ends the walk at its tile's end, for all lanes
            // at once: nothing before that branches on one lane's answer)
            ok = tc::mbar_wait(&ctl.q_full, 0, a.err, abort);
            tc::fence_proxy_async_smem();
            for (int i = 0; i < tiles; i++) {
                const uint32_t ph = i & 1;
                // What is behind the barriers was written through the generic
                // proxy (stores or cp.async); this warp's fence orders it before
                // the MMAs' reads (one fence here costs less than one in each
                // of the storing threads: 1007 against 1020 us at 1024 queries).
                for (int m = 0; m < mt; m++) {
                    ok &= tc::mbar_wait(&ctl.full[m], ph, a.err, abort);
                    tc::fence_proxy_async_smem();
                    tc::tc_fence_after();
                    const uint64_t kd = kd0 + m * (2 * kRegion / 16), qd = qd0 + m * (2 * NH * 128 / 16);
                    if (tc::elect_one()) {
#pragma unroll
                        for (int x = 0; x < 8; x++)
                            tc::mma_f16(tmem, kd + (x >> 2) * (kRegion / 16) + (x & 3) * 2,
                                        qd + (x >> 2) * (NH * 128 / 16) + (x & 3) * 2, id_qk, m > 0 || x > 0);
                    }
                    __syncwarp();
                }
                ok &= tc::mbar_wait(&ctl.full[4], ph, a.err, abort);
                tc::fence_proxy_async_smem();
                tc::tc_fence_after();
                if (tc::elect_one()) {
                    for (int x = 0; x < rope_steps; x++)
                        tc::mma_f16(tmem, kd0 + nc * (kRegion / 16) + x * 2, qd0 + nc * (NH * 128 / 16) + x * 2, id_qk,
                                    true);
                    tc::tc_commit(&ctl.s_done);
                }
                __syncwarp();
                if (i == 0 && !one_tile) {
                    tc::named_barrier(2, kThreads);
                    const int last = __shfl_sync(0xffffffffu, ctl.last, 0);
                    tiles = last < lo ? 1 : (last - lo) / kTile + 1;
                }
                ok &= tc::mbar_wait(&ctl.p_full, ph, a.err, abort);
                tc::fence_proxy_async_smem();
                tc::tc_fence_after();
                // step x: slots [16 x, 16 x + 16) of the chunk pair (A, two
                // 64-column atoms 16 KB apart) and of P (B), both MN-major
                if (tc::elect_one()) {
                    for (int m = 0; m < mt; m++) {
                        const uint64_t vd = vd0 + m * (2 * kRegion / 16);
#pragma unroll
                        for (int x = 0; x < kTile / 16; x++)
                            tc::mma_f16(tmem + NH * (m + 1), vd + x * (2048 / 16), pd0 + x * (2048 / 16), id_pv,
                                        i > 0 || x > 0);
                        tc::tc_commit(&ctl.o_done[m]);
                    }
                }
                if (!tc::warp_agrees(ok)) break;
            }
            // every issued MMA completes before TMEM is released, after a wait
            // that gave up too (this one does not look at the others' flag)
            if (tc::elect_one()) tc::tc_commit(&ctl.mma_fin);
            __syncwarp();
            int alone = 0;
            tc::mbar_wait(&ctl.mma_fin, 0, a.err, &alone);
        }
        __syncwarp();
    }
    // ------------------------------------------------------------ epilogue
    if (warp < kWork / 32) {
        // (none is in flight unless a wait gave up)
        asm volatile("cp.async.wait_all;" ::: "memory");
        tc::named_barrier(3, kWork);
        // thread = (column of dc, quarter of the heads): a warp stores 32
        // consecutive columns of one head at a time
        const int q4 = warp & 3, c = warp >> 2;
        if (c * kCols < NH) {
            for (int m = 0; m < mt; m++) {
                if (!tc::mbar_wait(&ctl.o_done[m], (tiles - 1) & 1, a.err, abort)) ok = false;
                tc::tc_fence_after();
                uint32_t v[kCols];
                ld_cols(tmem + ((uint32_t)(q4 * 32) << 16) + NH * (m + 1) + c * kCols, v);
                tc::tmem_wait_ld();
                const int col = m * 128 + q4 * 32 + lane;
                const int n = ok && !*abort ? heads - c * kCols : 0;   // heads of this thread
                if (a.splits > 1) {
                    float *o = a.part_o + ((int64_t)blockIdx.x * NH + c * kCols) * a.dc + col;
#pragma unroll
                    for (int e = 0; e < kCols; e++)
                        if (e < n) o[e * a.dc] = __uint_as_float(v[e]);
                } else {
                    __nv_bfloat16 *o = a.out + (row * a.Hq + h0 + c * kCols) * a.dc + col;
#pragma unroll
                    for (int e = 0; e < kCols; e++)
                        if (e < n) o[e * a.dc] = __float2bfloat16_rn(__uint_as_float(v[e]) * ctl.fac[c * kCols + e]);
                }
            }
        }
    }
    tc::tc_fence_before();
    __syncthreads();
    if (warp == kWork / 32) {
        tc::tc_fence_after();
        tc::tmem_dealloc(tmem, ncols);
    }
}

// Merges a row's splits: block = one head of one row, thread = four output
// columns.
//   M = max_s ref_s,  w_s = 2^(scale (ref_s - M)),  out = sum_s w_s O_s / sum_s w_s l_s
// Every warp works the splits' weights out for itself (lane = split), so that
// the partials' loads depend on two loads and no barrier; eight are in flight.
__global__ void __launch_bounds__(128)
latent_combine_kernel(const float *part_o, const float2 *part_ml, int splits, int groups, int nh, int Hq, int dc,
                      float scale, __nv_bfloat16 *out, float *lse) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int64_t row = blockIdx.x / (unsigned)Hq;
    const int head = (int)(blockIdx.x % (unsigned)Hq), lane = threadIdx.x & 31;
    const int64_t unit = (row * groups + head / kMaxHeads) * splits;
    const float2 *ml = part_ml + unit * nh + head % kMaxHeads;
    const float4 *o = reinterpret_cast<const float4 *>(part_o + (unit * nh + head % kMaxHeads) * dc) + threadIdx.x;
    const int64_t step = (int64_t)nh * dc / 4;             // float4s from split to split
    float M = -INFINITY;
    for (int s = lane; s < splits; s += 32) M = fmaxf(M, ml[(int64_t)s * nh].x);
    M = warp_max(M);
    float L = 0.f;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int s0 = 0; s0 < splits; s0 += 32) {
        // an empty share has l = 0 and a partial of zeros: weight 0, not read
        const float2 v = s0 + lane < splits ? ml[(int64_t)(s0 + lane) * nh] : make_float2(-INFINITY, 0.f);
        const float w = v.y == 0.f ? 0.f : v.x == M ? 1.f : ex2((v.x - M) * scale);
        const uint32_t live = __ballot_sync(0xffffffffu, v.y != 0.f);
        L += warp_sum(w == 0.f ? 0.f : w * v.y);
        const int n = splits - s0 < 32 ? splits - s0 : 32;
        for (int s1 = 0; s1 < n; s1 += 8) {
            float4 x[8];
#pragma unroll
            for (int u = 0; u < 8; u++)
                x[u] = live >> (s1 + u) & 1 ? o[(s0 + s1 + u) * step] : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int u = 0; u < 8; u++) {
                const float wu = __shfl_sync(0xffffffffu, w, s1 + u);
                acc.x = fmaf(wu, x[u].x, acc.x);
                acc.y = fmaf(wu, x[u].y, acc.y);
                acc.z = fmaf(wu, x[u].z, acc.z);
                acc.w = fmaf(wu, x[u].w, acc.w);
            }
        }
    }
    const float inv = L == 0.f ? 0.f : 1.f / L;
    uint2 w2;
    w2.x = bf16x2_bits(__floats2bfloat162_rn(acc.x * inv, acc.y * inv));
    w2.y = bf16x2_bits(__floats2bfloat162_rn(acc.z * inv, acc.w * inv));
    reinterpret_cast<uint2 *>(out + (row * Hq + head) * dc)[threadIdx.x] = w2;
    if (threadIdx.x == 0 && lse) lse[row * Hq + head] = L == 0.f ? -INFINITY : fmaf(M, scale, log2f(L)) * kLn2;
}

// How a call is cut: heads per CTA, head groups, splits of each row's slots.
struct Plan {
    int nh, groups, splits, split_slots;
    size_t o_bytes, total;
};

// (slots: up to 2^30, which leaves the kernel's slot numbers room in 32 bits)
Plan make_plan(int64_t rows, int Hq, int dc, int slots) {
    Plan p;
    // the MMA's N: a head count that fits 16 or 32 columns takes that many
    p.nh = Hq <= 16 ? 16 : Hq <= 32 ? 32 : kMaxHeads;
    p.groups = (Hq + p.nh - 1) / p.nh;
    const int64_t units = rows * p.groups;
    const int tiles = (slots + kTile - 1) / kTile;
    // one CTA per SM: split a row's tiles over the SMs that are left
    const int64_t share = units > 0 ? num_sms() / units : 1;
    int splits = share < 1 ? 1 : share < tiles ? (int)share : tiles;
    const int per = (tiles + splits - 1) / splits;
    p.splits = (tiles + per - 1) / per;
    p.split_slots = per * kTile;
    p.o_bytes = p.total = 0;
    if (p.splits > 1) {
        const size_t n = (size_t)units * p.splits * p.nh;
        p.o_bytes = align_up(n * dc * sizeof(float), 256);
        p.total = p.o_bytes + n * sizeof(float2);
    }
    return p;
}

int slots_of(int n_sel, int block) { return block ? (n_sel + 1) * block : n_sel; }

template <int F, int NH>
dsa_status launch_kernel(const AttnArgs &a, unsigned grid, cudaStream_t st) {
    const size_t smem = smem_bytes(a.dc, NH);
    if (cudaFuncSetAttribute(latent_attn_kernel<F, NH>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             (int)smem_bytes(512, NH)) != cudaSuccess)
        return DSA_ERR_CUDA;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    // programmatic: the set-up overlaps the preceding kernel's tail
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (cudaLaunchKernelEx(&cfg, latent_attn_kernel<F, NH>, a) != cudaSuccess) return DSA_ERR_CUDA;
    return launch_status();
}

template <int F>
dsa_status launch_heads(const AttnArgs &a, int nh, unsigned grid, cudaStream_t st) {
    return nh == 16   ? launch_kernel<F, 16>(a, grid, st)
           : nh == 32 ? launch_kernel<F, 32>(a, grid, st)
                      : launch_kernel<F, 64>(a, grid, st);
}

}  // namespace

size_t latent_attn_workspace_bytes(int B, int S, int Hq, int dc, int dr, int n_sel, int block) {
    (void)dr;
    return make_plan((int64_t)B * S, Hq, dc, slots_of(n_sel, block)).total;
}

dsa_status launch_latent_attn(const void *q, const void *kv, dsa_dtype fmt, int64_t t_max, const int32_t *sel,
                              int n_sel, int block, int B, int S, int Hq, int dc, int dr, int64_t start_pos,
                              float sm_scale, void *out, float *lse, void *ws, cudaStream_t st) {
    const int64_t rows = (int64_t)B * S;
    AttnArgs a = {};
    a.slots = slots_of(n_sel, block);
    const Plan p = make_plan(rows, Hq, dc, a.slots);
    a.q = static_cast<const __nv_bfloat16 *>(q);
    a.kv = static_cast<const uint8_t *>(kv);
    a.sel = sel;
    a.out = static_cast<__nv_bfloat16 *>(out);
    a.lse = lse;
    a.part_o = static_cast<float *>(ws);
    a.part_ml = reinterpret_cast<float2 *>(static_cast<char *>(ws) + p.o_bytes);
    a.t_max = t_max;
    a.start_pos = start_pos;
    a.row_bytes = latent_fmt_row_bytes(fmt, dc, dr);
    a.n_sel = n_sel;
    a.block = block;
    a.S = S;
    a.Hq = Hq;
    a.dc = dc;
    a.dr = dr;
    a.groups = p.groups;
    a.splits = p.splits;
    a.split_slots = p.split_slots;
    a.sign = copysignf(1.f, sm_scale);
    a.scale = fabsf(sm_scale) * kLog2e;
    if (a.scale < kLeastScale) a.scale = kLeastScale;
    a.err = device_error_word();
    const unsigned grid = (unsigned)(rows * p.groups * p.splits);
    const dsa_status s = fmt == DSA_BF16         ? launch_heads<DSA_BF16>(a, p.nh, grid, st)
                         : fmt == DSA_FP8_LATENT ? launch_heads<DSA_FP8_LATENT>(a, p.nh, grid, st)
                                                 : launch_heads<DSA_Q4_LATENT>(a, p.nh, grid, st);
    if (s != DSA_OK || p.splits == 1) return s;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(rows * Hq));
    cfg.blockDim = dim3((unsigned)(dc / 4));
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (cudaLaunchKernelEx(&cfg, latent_combine_kernel, (const float *)a.part_o, (const float2 *)a.part_ml,
                           p.splits, p.groups, p.nh, Hq, dc, a.scale, a.out, lse) != cudaSuccess)
        return DSA_ERR_CUDA;
    return launch_status();
}

namespace {

// The checks that both entry points share.  DSA_OK with *run = false: nothing to do.
dsa_status check_attn(const void *q, const void *kv, int64_t t_max, const int32_t *sel, int n_sel, int block,
                      int B, int S, int Hq, int dc, int dr, int64_t start_pos, const void *out, const float *lse,
                      const void *ws, size_t ws_bytes, bool *run) {
    *run = false;
    // (without a finished block there is none to list: the unfinished one is attended)
    if (B < 0 || S < 0 || Hq < 0 || n_sel < (block ? 0 : 1) || start_pos < 0) return DSA_ERR_INVALID_ARG;
    if (!latent_shape_ok(dc, dr)) return DSA_ERR_UNSUPPORTED;
    if (Hq > 1024 || block > 1 << 20) return DSA_ERR_UNSUPPORTED;
    if (B == 0 || S == 0 || Hq == 0) return DSA_OK;
    if (t_max > INT32_MAX || t_max < S || start_pos > t_max - S) return DSA_ERR_INVALID_ARG;
    if ((int64_t)B * S > INT32_MAX || (int64_t)B * S * Hq > INT32_MAX ||
        ((int64_t)n_sel + 1) * (block ? block : 1) > 1 << 30)
        return DSA_ERR_UNSUPPORTED;
    if (!q || !kv || (!sel && n_sel > 0) || !out) return DSA_ERR_INVALID_ARG;
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
    if (B <= 0 || S <= 0 || Hq <= 0 || k <= 0 || k >= 1 << 30 || !dsa::latent_shape_ok(dc, dr)) return 0;
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
    if (B <= 0 || S <= 0 || Hq <= 0 || kb < 0 || block <= 0 || !dsa::latent_shape_ok(dc, dr)) return 0;
    if (((int64_t)kb + 1) * block > 1 << 30) return 0;     // (the call refuses it)
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
