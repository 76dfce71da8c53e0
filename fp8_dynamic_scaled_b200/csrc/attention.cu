// attention.cu -- causal attention of bf16 queries over the paged FP8 cache (sm_100a).
//
//   out[t, h] = sum_j p_j v_j,  p = softmax_j(scale q[t, h] . k_j),  j up to t's own position
//
// One pass over the cached tokens with a running maximum and sum.  The heads that share a KV
// head are rows of one tile (rows = query tokens x group), so that a page is read once for
// all of them.  Operands of the products are fp16: FP8 codes are fp16 values (no rounding);
// a query row is first divided by a power of two so that its largest element is in [1, 2); the
// weights p are at most 2^15, so that fp16 keeps 11 bits of a weight down to 2^-29 of the
// largest.  Scores, softmax statistics and sums are fp32.
//
// The page's scales: with z = scale q . code_k * s_k in units of log2, the running maximum M is
// taken over z + log2 s_v, and the weight is w = 2^(z + log2 s_v - M + 15): sum w code_v is then
// sum p v without a product per page, whatever the spread of s_v among pages, and the sum of
// the softmax is sum w / s_v.
#include "kv_common.cuh"

namespace fp8b {

namespace {

constexpr int A_WARPS = 4;
constexpr int A_THREADS = 32 * A_WARPS;
constexpr int A_ROWS = 16;            // rows of a tile (mma m16)
constexpr int A_STEP = 32;            // tokens per warp and iteration
constexpr int A_CTA_STEP = A_STEP * A_WARPS;
constexpr float LOG2E = 1.4426950408889634f;
constexpr float P_SHIFT = 15.0f;

struct AttnParams {
    KvArgs c;
    const uint16_t* q;
    uint16_t* out;
    int64_t ldq, ldo, max_kv;
    int32_t q_heads, group;
    int32_t row_tiles;                // per (sequence, KV head)
    int32_t splits, chunk;            // tokens of one split (a multiple of A_CTA_STEP)
    float scale2;                     // softmax_scale * log2(e)
    float* part_o;                    // [units][splits][A_ROWS][D], unit = (b, head, row tile)
    float2* part_ml;                  // [units][splits][A_ROWS]: maximum (log2), sum
};

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// Two codes (the low 16 bits) -> two fp16 values, exactly.
template <int FMT>
__device__ __forceinline__ uint32_t half2_of(uint32_t codes2) {
    const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(codes2 & 0xFFFFu),
                                                    FMT == FP8_E4M3 ? __NV_E4M3 : __NV_E5M2);
    return (uint32_t)h.x | ((uint32_t)h.y << 16);
}
__device__ __forceinline__ uint32_t pack_half2(float a, float b) {
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ float quad_max(float v) {
    v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 1));
    return fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 2));
}
__device__ __forceinline__ float quad_sum(float v) {
    v += __shfl_xor_sync(0xffffffffu, v, 1);
    return v + __shfl_xor_sync(0xffffffffu, v, 2);
}

// The rows of one tile and the tokens that they see together.
struct Tile {
    int32_t b, head, row0, rows;      // rows of the sequence and head in all
    int32_t see;                      // tokens the last row of the tile sees
    Sequence s;
};

__device__ __forceinline__ Tile tile_of(const AttnParams& p, int32_t unit) {
    Tile t;
    const int32_t rt = unit % p.row_tiles, bh = unit / p.row_tiles;
    t.head = bh % p.c.kv_heads;
    t.b = bh / p.c.kv_heads;
    t.s = sequence_of(p.c, t.b, p.max_kv);
    t.row0 = rt * A_ROWS;
    t.rows = t.s.n * p.group;
    const int32_t last = min(t.row0 + A_ROWS, t.rows) - 1;
    t.see = last >= t.row0 ? max(0, t.s.kv_len - t.s.n + last / p.group + 1) : 0;
    return t;
}

// ---------------------------------------------------------------- the split kernel
// Fragment layouts (c = lane % 4, r = lane / 4).  QK: the reduction index is permuted so
// that a lane's operands are 16 contiguous bytes of a token's K row: k-step kk takes the 4
// codes at (kk / 4) * 64 + 16 c + 4 (kk % 4).  PV: n-tile j of the output holds
// d = (D / 8) n + j, so that a lane's operands are D / 8 contiguous bytes of a V row.
template <int FMT, int D>
__global__ void __launch_bounds__(A_THREADS, 2) kv_attention_kernel(const __grid_constant__ AttnParams p) {
    constexpr int KK = D / 16;                 // k-steps of QK = n-tiles of K's 16-byte chunks * 4
    constexpr int NT = D / 8;                  // n-tiles of PV
    constexpr int CH = D / 64;                 // 16-byte chunks of a K row per lane
    __shared__ float so[A_WARPS][A_ROWS][D];
    __shared__ float2 sml[A_WARPS][A_ROWS];
    const int32_t unit = (int32_t)(blockIdx.x / p.splits), split = (int32_t)(blockIdx.x % p.splits);
    const Tile t = tile_of(p, unit);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, c = lane & 3, r = lane >> 2;
    if (!t.s.ok) {
        if (split == 0 && threadIdx.x == 0) report_status(p.c.status, FP8_ERR_INVALID_ARG);
        return;
    }
    if (t.row0 >= t.rows) return;
    const int32_t begin = split * p.chunk, end = min(t.see, begin + p.chunk);
    const int32_t used = max(1, (t.see + p.chunk - 1) / p.chunk);       // splits with tokens
    if (split >= used) return;
    const int32_t P = p.c.page_size;
    // ---- the tile's rows: r and r + 8
    int32_t limit[2];                           // tokens the row sees (0: a row beyond the last)
    uint32_t qa[KK][4];
    float qf[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int32_t row = t.row0 + r + 8 * i;
        const bool real = row < t.rows;
        const int32_t tok = real ? row / p.group : 0;
        limit[i] = real ? max(0, t.s.kv_len - t.s.n + tok + 1) : 0;
        const uint16_t* src = p.q + (int64_t)(t.s.first + tok) * p.ldq +
                              (int64_t)(t.head * p.group + (real ? row % p.group : 0)) * D;
        uint4 v[CH][2];
        uint32_t m2 = 0;
#pragma unroll
        for (int h = 0; h < CH; ++h)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                v[h][e] = real ? ld_v4(src + h * 64 + 16 * c + 8 * e) : make_uint4(0, 0, 0, 0);
                m2 = max_bf16x2_bits(m2, max_bf16x2_bits(max_bf16x2_bits(abs_bf16x2(v[h][e].x), abs_bf16x2(v[h][e].y)),
                                                         max_bf16x2_bits(abs_bf16x2(v[h][e].z), abs_bf16x2(v[h][e].w))));
            }
        uint32_t m = hmax_pair(m2);
        m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
        m = max(m, __shfl_xor_sync(0xffffffffu, m, 2));
        const int e = max(1, min((int)(m >> 7), 253));                  // biased exponent of the row's largest
        const float inv = __uint_as_float((uint32_t)(254 - e) << 23);   // 2^(127 - e)
        qf[i] = __uint_as_float((uint32_t)e << 23) * p.scale2;
#pragma unroll
        for (int h = 0; h < CH; ++h)
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const uint32_t w0 = k < 2 ? (k == 0 ? v[h][0].x : v[h][0].z) : (k == 2 ? v[h][1].x : v[h][1].z);
                const uint32_t w1 = k < 2 ? (k == 0 ? v[h][0].y : v[h][0].w) : (k == 2 ? v[h][1].y : v[h][1].w);
                qa[4 * h + k][i] = pack_half2(bf16_lo(w0) * inv, bf16_hi(w0) * inv);
                qa[4 * h + k][2 + i] = pack_half2(bf16_lo(w1) * inv, bf16_hi(w1) * inv);
            }
    }
    const int32_t least = max(0, t.s.kv_len - t.s.n + t.row0 / p.group + 1);   // tokens the first row sees
    float o[NT][4];
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[j][e] = 0.0f;
    float mrow[2] = {-INFINITY, -INFINITY}, lrow[2] = {0.0f, 0.0f};

    // ---- pages: lane i holds the place of the 16 tokens i % 2 of iteration i / 2 of this warp
    int32_t pages_at = -16;                     // first iteration that the lanes hold
    int64_t place = -1;
    float ksc = 0.0f, vsc = 0.0f;
    const int32_t iters = end > begin ? (end - begin + A_CTA_STEP - 1) / A_CTA_STEP : 0;
    auto hold = [&](int32_t it) {
        if (it < pages_at + 16) return;
        pages_at = it;
        const int32_t tok = begin + (it + (lane >> 1)) * A_CTA_STEP + warp * A_STEP + (lane & 1) * 16;
        place = -1;
        ksc = vsc = 1.0f;
        if (tok < end) {
            const int32_t page = __ldg(p.c.table + (int64_t)t.b * p.c.table_stride + tok / P);
            if (page >= 0 && page < p.c.num_pages) {
                const int64_t at = (int64_t)page * p.c.kv_heads + t.head;
                place = (at * P + tok % P) * D;
                ksc = __ldg(p.c.k_scale + at);
                vsc = __ldg(p.c.v_scale + at);
            } else {
                report_status(p.c.status, FP8_ERR_INVALID_ARG);
            }
        }
    };
    uint4 kb[4][CH];                            // K of 32 tokens: token 8 i + r, chunks
    uint2 vb[8][NT / 8];                        // V of 32 tokens: 16 (i / 4) + {2c, 2c+1, 2c+8, 2c+9}[i % 4]
    auto load_k = [&](int32_t it) {
#pragma unroll
        for (int g = 0; g < 2; ++g) {
            const int64_t at = __shfl_sync(0xffffffffu, place, ((it - pages_at) << 1) + g);
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int h = 0; h < CH; ++h) {
                    kb[2 * g + i][h] = make_uint4(0, 0, 0, 0);
                    if (at >= 0) kb[2 * g + i][h] = ld_v4_stream(p.c.k + at + (8 * i + r) * D + h * 64 + 16 * c);
                }
        }
    };
    auto load_v = [&](int32_t it) {
#pragma unroll
        for (int g = 0; g < 2; ++g) {
            const int64_t at = __shfl_sync(0xffffffffu, place, ((it - pages_at) << 1) + g);
            const int32_t left = end - (begin + it * A_CTA_STEP + warp * A_STEP + 16 * g);   // tokens of the group
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int tok = 2 * c + (i & 1) + 8 * (i >> 1);
                // slots past the last token may hold anything: they count as zeros
                const bool in = at >= 0 && tok < left;
                const uint8_t* src = p.c.v + (in ? at : 0) + tok * D + r * NT;
                if (NT == 16) {
                    uint4 v = make_uint4(0, 0, 0, 0);
                    if (in) v = ld_v4_stream(src);
                    vb[4 * g + i][0] = make_uint2(v.x, v.y);
                    vb[4 * g + i][NT / 8 - 1] = make_uint2(v.z, v.w);
                } else {
                    vb[4 * g + i][0] = make_uint2(0, 0);
                    if (in) vb[4 * g + i][0] = __ldcs(reinterpret_cast<const uint2*>(src));
                }
            }
        }
    };
    if (iters > 0) {
        hold(0);
        load_k(0);
        load_v(0);
    }
    for (int32_t it = 0; it < iters; ++it) {
        const int32_t tok0 = begin + it * A_CTA_STEP + warp * A_STEP;
        const float ks[2] = {__shfl_sync(0xffffffffu, ksc, ((it - pages_at) << 1)),
                             __shfl_sync(0xffffffffu, ksc, ((it - pages_at) << 1) + 1)};
        const float vs[2] = {__shfl_sync(0xffffffffu, vsc, ((it - pages_at) << 1)),
                             __shfl_sync(0xffffffffu, vsc, ((it - pages_at) << 1) + 1)};
        const int64_t pl[2] = {__shfl_sync(0xffffffffu, place, ((it - pages_at) << 1)),
                               __shfl_sync(0xffffffffu, place, ((it - pages_at) << 1) + 1)};
        // ---- scores
        float s[4][4];
#pragma unroll
        for (int n = 0; n < 4; ++n) {
#pragma unroll
            for (int e = 0; e < 4; ++e) s[n][e] = 0.0f;
#pragma unroll
            for (int h = 0; h < CH; ++h) {
                const uint32_t w[4] = {kb[n][h].x, kb[n][h].y, kb[n][h].z, kb[n][h].w};
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    mma16816(s[n], qa[4 * h + k], half2_of<FMT>(w[k]), half2_of<FMT>(w[k] >> 16));
            }
        }
        if (it + 1 < iters) {
            hold(it + 1);
            load_k(it + 1);
        }
        // ---- weights
        float lv[2], iv[2];
#pragma unroll
        for (int g = 0; g < 2; ++g) {
            lv[g] = __log2f(vs[g]) + P_SHIFT;
            iv[g] = __frcp_rn(vs[g]);
        }
        const bool edge = tok0 + A_STEP > least || pl[0] < 0 || pl[1] < 0;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            float top = -INFINITY;
#pragma unroll
            for (int n = 0; n < 4; ++n) {
                const float f = qf[i] * ks[n >> 1];
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    float z = fmaf(s[n][2 * i + e], f, lv[n >> 1]);
                    if (edge && (tok0 + 8 * n + 2 * c + e >= min(limit[i], end) || pl[n >> 1] < 0)) z = -INFINITY;
                    s[n][2 * i + e] = z;
                    top = fmaxf(top, z);
                }
            }
            top = quad_max(top);
            const float m_new = fmaxf(mrow[i], top - P_SHIFT);
            const float base = m_new == -INFINITY ? 0.0f : m_new;
            const float corr = ex2(mrow[i] - base);
            mrow[i] = m_new;
            float sum = 0.0f;
#pragma unroll
            for (int g = 0; g < 2; ++g) {
                float part = 0.0f;
#pragma unroll
                for (int n = 2 * g; n < 2 * g + 2; ++n)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const float w = ex2(s[n][2 * i + e] - base);
                        s[n][2 * i + e] = w;
                        part += w;
                    }
                sum = fmaf(part, iv[g], sum);
            }
            lrow[i] = fmaf(lrow[i], corr, sum);
            if (__any_sync(0xffffffffu, corr != 1.0f)) {
#pragma unroll
                for (int j = 0; j < NT; ++j) {
                    o[j][2 * i] *= corr;
                    o[j][2 * i + 1] *= corr;
                }
            }
        }
        // ---- the values
#pragma unroll
        for (int g = 0; g < 2; ++g) {
            const uint32_t a[4] = {pack_half2(s[2 * g][0], s[2 * g][1]), pack_half2(s[2 * g][2], s[2 * g][3]),
                                   pack_half2(s[2 * g + 1][0], s[2 * g + 1][1]),
                                   pack_half2(s[2 * g + 1][2], s[2 * g + 1][3])};
#pragma unroll
            for (int q = 0; q < NT / 4; ++q) {
                uint32_t w[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) w[i] = (q & 1) ? vb[4 * g + i][q >> 1].y : vb[4 * g + i][q >> 1].x;
                const uint32_t lo0 = __byte_perm(w[0], w[1], 0x5140), hi0 = __byte_perm(w[0], w[1], 0x7362);
                const uint32_t lo1 = __byte_perm(w[2], w[3], 0x5140), hi1 = __byte_perm(w[2], w[3], 0x7362);
                mma16816(o[4 * q + 0], a, half2_of<FMT>(lo0), half2_of<FMT>(lo1));
                mma16816(o[4 * q + 1], a, half2_of<FMT>(lo0 >> 16), half2_of<FMT>(lo1 >> 16));
                mma16816(o[4 * q + 2], a, half2_of<FMT>(hi0), half2_of<FMT>(hi1));
                mma16816(o[4 * q + 3], a, half2_of<FMT>(hi0 >> 16), half2_of<FMT>(hi1 >> 16));
            }
        }
        if (it + 1 < iters) load_v(it + 1);
    }
    // ---- join the warps
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        lrow[i] = quad_sum(lrow[i]);
        if (c == 0) sml[warp][r + 8 * i] = make_float2(mrow[i], lrow[i]);
    }
    __syncthreads();
    float keep[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        float m = -INFINITY;
#pragma unroll
        for (int w = 0; w < A_WARPS; ++w) m = fmaxf(m, sml[w][r + 8 * i].x);
        keep[i] = m == -INFINITY ? 0.0f : ex2(mrow[i] - m);
    }
#pragma unroll
    for (int e = 0; e < 4; ++e)
#pragma unroll
        for (int j = 0; j < NT; j += 4)
            *reinterpret_cast<float4*>(&so[warp][r + 8 * (e >> 1)][NT * (2 * c + (e & 1)) + j]) =
                make_float4(o[j][e] * keep[e >> 1], o[j + 1][e] * keep[e >> 1], o[j + 2][e] * keep[e >> 1],
                            o[j + 3][e] * keep[e >> 1]);
    __syncthreads();
    for (int32_t k = threadIdx.x; k < A_ROWS * D / 8; k += A_THREADS) {
        const int32_t row = k / (D / 8), d = (k % (D / 8)) * 8;
        if (t.row0 + row >= t.rows) continue;
        float m = -INFINITY, l = 0.0f;
#pragma unroll
        for (int w = 0; w < A_WARPS; ++w) m = fmaxf(m, sml[w][row].x);
#pragma unroll
        for (int w = 0; w < A_WARPS; ++w)
            if (m != -INFINITY) l = fmaf(sml[w][row].y, ex2(sml[w][row].x - m), l);
        float v[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            v[e] = 0.0f;
#pragma unroll
            for (int w = 0; w < A_WARPS; ++w) v[e] += so[w][row][d + e];
        }
        if (used == 1) {
            const float inv = l > 0.0f ? __frcp_rn(l) : 0.0f;
            uint16_t* dst = p.out + (int64_t)(t.s.first + (t.row0 + row) / p.group) * p.ldo +
                            (int64_t)(t.head * p.group + (t.row0 + row) % p.group) * D + d;
            *reinterpret_cast<uint4*>(dst) =
                make_uint4(pack_bf16x2(v[0] * inv, v[1] * inv), pack_bf16x2(v[2] * inv, v[3] * inv),
                           pack_bf16x2(v[4] * inv, v[5] * inv), pack_bf16x2(v[6] * inv, v[7] * inv));
        } else {
            const int64_t at = ((int64_t)unit * p.splits + split) * A_ROWS + row;
            float4* dst = reinterpret_cast<float4*>(p.part_o + at * D + d);
            dst[0] = make_float4(v[0], v[1], v[2], v[3]);
            dst[1] = make_float4(v[4], v[5], v[6], v[7]);
            if (d == 0) p.part_ml[at] = make_float2(m, l);
        }
    }
}

// ---------------------------------------------------------------- the joining kernel
// One thread per 8 elements of a row; nothing to do for rows that one split covered.
template <int D>
__global__ void __launch_bounds__(A_ROWS * D / 8) kv_attention_join_kernel(const __grid_constant__ AttnParams p) {
    const int32_t unit = (int32_t)blockIdx.x;
    const Tile t = tile_of(p, unit);
    if (!t.s.ok || t.row0 >= t.rows) return;
    const int32_t used = (t.see + p.chunk - 1) / p.chunk;
    if (used <= 1) return;
    const int32_t row = threadIdx.x / (D / 8), d = (threadIdx.x % (D / 8)) * 8;
    if (t.row0 + row >= t.rows) return;
    const int64_t at = (int64_t)unit * p.splits * A_ROWS + row;
    float m = -INFINITY;
    for (int32_t s = 0; s < used; ++s) m = fmaxf(m, p.part_ml[at + (int64_t)s * A_ROWS].x);
    float l = 0.0f, v[8] = {};
    if (m != -INFINITY) {
        for (int32_t s = 0; s < used; ++s) {
            const float2 ml = p.part_ml[at + (int64_t)s * A_ROWS];
            const float f = ex2(ml.x - m);
            l = fmaf(ml.y, f, l);
            const float4* src = reinterpret_cast<const float4*>(p.part_o + (at + (int64_t)s * A_ROWS) * D + d);
            const float4 a = src[0], b = src[1];
            v[0] = fmaf(a.x, f, v[0]); v[1] = fmaf(a.y, f, v[1]); v[2] = fmaf(a.z, f, v[2]); v[3] = fmaf(a.w, f, v[3]);
            v[4] = fmaf(b.x, f, v[4]); v[5] = fmaf(b.y, f, v[5]); v[6] = fmaf(b.z, f, v[6]); v[7] = fmaf(b.w, f, v[7]);
        }
    }
    const float inv = l > 0.0f ? __frcp_rn(l) : 0.0f;
    uint16_t* dst = p.out + (int64_t)(t.s.first + (t.row0 + row) / p.group) * p.ldo +
                    (int64_t)(t.head * p.group + (t.row0 + row) % p.group) * D + d;
    *reinterpret_cast<uint4*>(dst) = make_uint4(pack_bf16x2(v[0] * inv, v[1] * inv), pack_bf16x2(v[2] * inv, v[3] * inv),
                                                pack_bf16x2(v[4] * inv, v[5] * inv), pack_bf16x2(v[6] * inv, v[7] * inv));
}

// How the cached tokens are split: enough CTAs for about four waves of two per SM, and no
// split shorter than 512 tokens (its partial result would cost more than it gives).
struct Plan {
    int64_t units;
    int32_t row_tiles, splits, chunk;
};
Plan plan_of(int32_t batch, int32_t q_heads, int32_t kv_heads, int32_t max_q, int64_t max_kv) {
    Plan pl;
    const int64_t rows = (int64_t)max_q * (q_heads / kv_heads);
    pl.row_tiles = (int32_t)((rows + A_ROWS - 1) / A_ROWS);
    pl.units = (int64_t)batch * kv_heads * pl.row_tiles;
    const int64_t want = std::max<int64_t>(1, 1184 / std::max<int64_t>(1, pl.units));
    int64_t chunk = std::max<int64_t>(512, (max_kv + want - 1) / want);
    chunk = (chunk + A_CTA_STEP - 1) / A_CTA_STEP * A_CTA_STEP;
    pl.chunk = (int32_t)chunk;
    pl.splits = (int32_t)std::max<int64_t>(1, (max_kv + chunk - 1) / chunk);
    return pl;
}

template <int FMT, int D>
cudaError_t launch_attention(const AttnParams& p, int64_t units, cudaStream_t st) {
    kv_attention_kernel<FMT, D><<<(unsigned)(units * p.splits), A_THREADS, 0, st>>>(p);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess || p.splits == 1) return e;
    kv_attention_join_kernel<D><<<(unsigned)units, A_ROWS * D / 8, 0, st>>>(p);
    return cudaGetLastError();
}

}  // namespace

size_t attention_workspace(int32_t batch, int32_t q_heads, int32_t kv_heads, int32_t head_dim, int32_t max_q,
                           int64_t max_kv) {
    const Plan pl = plan_of(batch, q_heads, kv_heads, max_q, max_kv);
    if (pl.splits == 1) return 0;
    return (size_t)pl.units * pl.splits * A_ROWS * (head_dim + 2) * sizeof(float);
}

cudaError_t launch_kv_attention(const AttnArgs& a, cudaStream_t st) {
    const Plan pl = plan_of(a.c.batch, a.q_heads, a.c.kv_heads, a.c.max_q, a.max_kv);
    if (pl.units * pl.splits >= ((int64_t)1 << 31)) return cudaErrorInvalidConfiguration;
    AttnParams p{};
    p.c = a.c;
    p.q = a.q;
    p.out = a.out;
    p.ldq = a.ldq;
    p.ldo = a.ldo;
    p.max_kv = a.max_kv;
    p.q_heads = a.q_heads;
    p.group = a.q_heads / a.c.kv_heads;
    p.row_tiles = pl.row_tiles;
    p.splits = pl.splits;
    p.chunk = pl.chunk;
    p.scale2 = a.softmax_scale * LOG2E;
    p.part_o = static_cast<float*>(a.workspace);
    p.part_ml = reinterpret_cast<float2*>(p.part_o + pl.units * pl.splits * A_ROWS * a.c.head_dim);
    if (a.c.fmt == FP8_E4M3)
        return a.c.head_dim == 128 ? launch_attention<FP8_E4M3, 128>(p, pl.units, st)
                                   : launch_attention<FP8_E4M3, 64>(p, pl.units, st);
    return a.c.head_dim == 128 ? launch_attention<FP8_E5M2, 128>(p, pl.units, st)
                               : launch_attention<FP8_E5M2, 64>(p, pl.units, st);
}

}  // namespace fp8b
