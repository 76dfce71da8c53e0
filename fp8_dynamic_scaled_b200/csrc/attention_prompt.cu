// attention_prompt.cu -- fp8_kv_attention for many query tokens: prompts and chunks of them
// (sm_100a).  attention.cu states the mathematics and holds the kernel for few rows.
//
// With many rows the products bound it: 4 D FLOP for each row and token that it sees, at the
// fp16 tensor rate.  A CTA owns 256 rows (query tokens x group) of one sequence and KV head as
// two tiles of 128 (the tensor core's M), and walks the cached tokens 128 at a time:
//   S = Q K^T    tcgen05.mma, Q and K in shared memory, S in tensor memory (128 columns)
//   W = weights  one thread per row reads its 128 scores, keeps the running maximum and sum
//                in registers (no exchange between threads), and writes W as fp16 over S
//   O += W V     tcgen05.mma, W from tensor memory, V from shared memory, O in tensor memory
// The two tiles take turns: while one's weights are computed the other's products run.
// Four warps turn FP8 codes into fp16 tiles in shared memory (exact), a tile ahead; both
// products read the same [64 elements][tokens] layout, K as its K-major and V as its
// MN-major operand.  O is moved to a new maximum only when a score passes the old one by 2^7
// (its products are then complete: they were issued before the scores' whose barrier the
// thread has waited for).
//
// Measured: three chunks (2048 new tokens of 6001, 587 of 3535, 512 of 4546; 32 / 8 heads of 128)
// 310 us = 755 TFLOP/s, a step of both tiles in some 4,900 cycles.  The products alone would take
// 2,048; the chain scores -> weights -> output of each tile bounds it (2,000-2,400 cycles for the
// weights, 1,400 for a tile's two products, the hand-overs): without the exponentials it is 2 %
// faster, without the loads 10 %, without either product 5 %.
//
// Roles: warp 0 issues the MMAs; warps 4-7 convert; warps 8-11 and 12-15 hold the rows.
#include "attention_common.cuh"

namespace fp8b {

namespace {

constexpr int T_ROWS = 128;                 // rows of a tile
constexpr int T_CTA_ROWS = 2 * T_ROWS;
constexpr int T_TOK = 128;                  // tokens of a step
constexpr int T_THREADS = 512;
constexpr int T_GROUPS = T_TOK / 16;        // a page holds at least 16 tokens
constexpr int T_HEADER = 1024;
constexpr uint32_t T_BLOCK = T_TOK * 128;   // 64 fp16 elements of 128 rows: 128-byte swizzled rows

template <int D>
constexpr uint32_t tile_bytes() { return (D / 64) * T_BLOCK; }
template <int D>
constexpr uint32_t prompt_smem() { return 1024 + T_HEADER + 6 * tile_bytes<D>(); }   // Q 2, K 2, V 2

struct Bars {
    uint64_t kfull[2], kempty[2], vfull[2], vempty[2], sfull[2], pfull[2], ofull[2], qfull, teardown;
    uint32_t tmem_slot;
    int32_t abort_flag;
};

// Per 16 tokens of a step: s_k, log2 s_v + P_SHIFT (-inf: no token there), 1 / s_v.
struct __align__(16) GroupInfo {
    float ks, lv, iv, pad;
};

__device__ __forceinline__ uint32_t swizzled(uint32_t row, uint32_t chunk) { return row * 128 + ((chunk ^ (row & 7)) << 4); }

// Shared-memory descriptor of an MN-major operand in the 128-byte swizzle: 128-byte rows of 64 MN
// elements, one row per K index; 8 rows (1024 B) to the next K group, `mn_stride` bytes to the
// next 64 MN elements.
__device__ __forceinline__ uint64_t sdesc_mnmajor_sw128(uint32_t smem_addr, uint32_t mn_stride) {
    return (uint64_t)((smem_addr >> 4) & 0x3FFFu) | ((uint64_t)(mn_stride >> 4) << 16) | ((uint64_t)(1024 >> 4) << 32) |
           ((uint64_t)1 << 46) | ((uint64_t)2 << 61);
}

// A wait that all lanes of a warp leave with the same outcome.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, Bars* bars, const AttnParams& p) {
    const bool ok = wait_limited(bar, parity, &bars->abort_flag, p.c.status, p.wait_ns);
    return __all_sync(0xffffffffu, ok);
}

struct Unit {
    int32_t h, row0, rows, sees;            // rows: of the sequence and head in all; sees: tokens of the CTA's last row
    Sequence s;
    int32_t b;
    int32_t steps[2];                       // of the two tiles
};

__device__ __forceinline__ int32_t sees_upto(const AttnParams& p, const Sequence& s, int32_t row) {
    return max(0, s.kv_len - s.n + row / p.group + 1);
}

// ---------------------------------------------------------------- the converters
// A step's K (or V) codes in the four warps' registers: a thread takes one 16-byte chunk of every
// 16th (D = 64: 32nd) row.  Eight neighbouring lanes take four chunks (64 elements) of two rows, so that
// both their loads (64 contiguous bytes) and their swizzled stores (all banks once) are whole.
template <int FMT, int D>
struct Codes {
    static constexpr int STEP = 128 * 16 / D;                   // rows between a thread's chunks
    static constexpr int N = T_TOK / STEP;                      // chunks per thread
    uint4 v[N];

    static __device__ __forceinline__ int32_t chunk(int32_t t) { return (t & 3) + (D == 128 ? 4 * ((t >> 3) & 1) : 0); }
    static __device__ __forceinline__ int32_t row0(int32_t t) {
        return D == 128 ? ((t >> 4) << 1) + ((t >> 2) & 1) : t >> 2;
    }

    // `at`: the first of 16 rows of codes in units of 16, -1 for none, in the lane first + their number in
    // the step; rows at or past `left` are zeros (those slots may hold anything).
    __device__ __forceinline__ void load(const uint8_t* base, int32_t at, int32_t first, int32_t t, int32_t left) {
        const int32_t r0 = row0(t);
        const uint8_t* mine = base + (r0 & 15) * D + chunk(t) * 16;
        const bool whole = left >= T_TOK &&
                           ((__ballot_sync(0xffffffffu, at >= 0) >> first) & ((1u << T_GROUPS) - 1)) == (1u << T_GROUPS) - 1;
        if (whole) {
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const int32_t g = __shfl_sync(0xffffffffu, at, first + (r0 >> 4) + i * (STEP / 16));
                v[i] = ld_v4(mine + (int64_t)g * (16 * D));
            }
        } else {
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const int32_t g = __shfl_sync(0xffffffffu, at, first + (r0 >> 4) + i * (STEP / 16));
                v[i] = make_uint4(0, 0, 0, 0);
                if (g >= 0 && r0 + STEP * i < left) v[i] = ld_v4(mine + (int64_t)g * (16 * D));
            }
        }
    }
    __device__ __forceinline__ void store(uint8_t* tile, int32_t t) const {
        const int32_t c = chunk(t), r0 = row0(t);                // r0 + STEP i has the same low three bits
        uint8_t* dst = tile + (c >> 2) * T_BLOCK + r0 * 128;
        const uint32_t o0 = (((c & 3) * 2) ^ (r0 & 7)) << 4, o1 = o0 ^ 16;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            uint4 lo, hi;
            half2x2_of<FMT>(v[i].x, lo.x, lo.y);
            half2x2_of<FMT>(v[i].y, lo.z, lo.w);
            half2x2_of<FMT>(v[i].z, hi.x, hi.y);
            half2x2_of<FMT>(v[i].w, hi.z, hi.w);
            *reinterpret_cast<uint4*>(dst + o0 + i * STEP * 128) = lo;
            *reinterpret_cast<uint4*>(dst + o1 + i * STEP * 128) = hi;
        }
    }
};

template <int FMT, int D>
__device__ __forceinline__ void convert(const AttnParams& p, const Unit& u, uint8_t* k16, uint8_t* v16, GroupInfo (*info)[T_GROUPS],
                                        Bars* bars) {
    const int32_t t = threadIdx.x - 128, lane = t & 31;
    const int32_t P = p.c.page_size;
    const int32_t steps = max(u.steps[0], u.steps[1]);
    // Lane i holds the place and the scales of 16 tokens of 4 steps: those of number i % 8 in step
    // 4 B + i / 8 of batch B; the pages of the next batch are on the way meanwhile.
    int32_t next_page = -1;
    int32_t place = -1;                       // in units of 16 rows of codes
    float ks = 0.0f, vs = 1.0f;
    auto fetch = [&](int32_t batch) {
        const int32_t tok = 16 * (32 * batch + lane);
        next_page = -1;
        if (tok < u.sees) next_page = __ldg(p.c.table + (int64_t)u.b * p.c.table_stride + tok / P);
    };
    auto take = [&](int32_t batch) {
        const int32_t tok = 16 * (32 * batch + lane);
        place = -1;
        ks = 0.0f;
        vs = 1.0f;
        if (tok < u.sees) {
            if (next_page >= 0 && next_page < p.c.num_pages) {
                const int64_t at = (int64_t)next_page * p.c.kv_heads + u.h;
                place = (int32_t)((at * P + tok % P) >> 4);
                ks = __ldg(p.c.k_scale + at);
                vs = __ldg(p.c.v_scale + at);
            } else {
                report_status(p.c.status, FP8_ERR_INVALID_ARG);
            }
        }
        __syncwarp();
        fetch(batch + 1);
        if (!v_scale_ok(vs)) report_status(p.c.status, FP8_ERR_INVALID_ARG);
    };
    Codes<FMT, D> k, v;
    fetch(0);
    take(0);
    k.load(p.c.k, place, 0, t, u.sees);
    for (int32_t j = 0; j < steps; ++j) {
        const int32_t buf = j & 1, first = (j & 3) * T_GROUPS;
        const uint32_t parity = ((j >> 1) & 1) ^ 1;
        v.load(p.c.v, place, first, t, u.sees - j * T_TOK);
        if (!warp_wait(&bars->kempty[buf], parity, bars, p)) return;
        k.store(k16 + buf * tile_bytes<D>(), t);
        if (t >= first && t < first + T_GROUPS) {          // warp 4's lanes of this step
            GroupInfo gi;
            gi.ks = ks;
            gi.lv = place >= 0 ? __log2f(vs) + P_SHIFT : -INFINITY;
            gi.iv = __frcp_rn(vs);
            gi.pad = 0.0f;
            info[j & 3][t - first] = gi;
        }
        ptx::fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(&bars->kfull[buf]);
        if (j + 1 < steps) {
            if (((j + 1) & 3) == 0) take((j + 1) >> 2);
            k.load(p.c.k, place, ((j + 1) & 3) * T_GROUPS, t, u.sees - (j + 1) * T_TOK);
        }
        if (!warp_wait(&bars->vempty[buf], parity, bars, p)) return;
        v.store(v16 + buf * tile_bytes<D>(), t);
        ptx::fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(&bars->vfull[buf]);
    }
}

// ---------------------------------------------------------------- the MMA issuer
template <int D>
__device__ __forceinline__ void issue(const AttnParams& p, const Unit& u, uint32_t q16, uint32_t k16, uint32_t v16,
                                      uint32_t tmem, Bars* bars) {
    // fp16 operands, fp32 accumulator, M = 128; scores: N = 128 tokens, both K-major; output: N = D,
    // V MN-major (bit 16)
    constexpr uint32_t idesc_s = (1u << 4) | ((uint32_t)(T_TOK >> 3) << 17) | ((uint32_t)(T_ROWS >> 4) << 24);
    constexpr uint32_t idesc_o = (1u << 4) | (1u << 16) | ((uint32_t)(D >> 3) << 17) | ((uint32_t)(T_ROWS >> 4) << 24);
    const int32_t steps = max(u.steps[0], u.steps[1]);
    auto scores = [&](int i, int32_t buf) {
#pragma unroll
        for (int k = 0; k < D / 16; ++k) {
            const uint32_t at = (k >> 2) * T_BLOCK + (k & 3) * 32;
            ptx::mma_f16(tmem + i * T_TOK, ptx::sdesc_kmajor_sw128(q16 + i * tile_bytes<D>() + at),
                         ptx::sdesc_kmajor_sw128(k16 + buf * tile_bytes<D>() + at), idesc_s, k != 0);
        }
        ptx::mma_commit(&bars->sfull[i]);
    };
    auto output = [&](int i, int32_t buf, bool more) {
#pragma unroll
        for (int k = 0; k < T_TOK / 16; ++k)
            ptx::mma_f16_ts(tmem + 2 * T_TOK + i * D, tmem + i * T_TOK + k * 8,
                            sdesc_mnmajor_sw128(v16 + buf * tile_bytes<D>() + k * 16 * 128, T_BLOCK), idesc_o, more || k != 0);
    };
    bool ok = warp_wait(&bars->qfull, 0, bars, p) && warp_wait(&bars->kfull[0], 0, bars, p);
    if (ok) {
        ptx::tc_fence_after();
        if (ptx::elect_one()) {
            scores(0, 0);
            if (u.steps[1] > 0) scores(1, 0);
            ptx::mma_commit(&bars->kempty[0]);
        }
        __syncwarp();
    }
    for (int32_t j = 0; j < steps && ok; ++j) {
        const int32_t buf = j & 1, nbuf = buf ^ 1;
        ok = warp_wait(&bars->vfull[buf], (j >> 1) & 1, bars, p);
        if (ok && j + 1 < steps) ok = warp_wait(&bars->kfull[nbuf], ((j + 1) >> 1) & 1, bars, p);
#pragma unroll 1
        for (int i = 0; i < 2 && ok; ++i) {
            if (j >= u.steps[i]) continue;
            ok = warp_wait(&bars->pfull[i], j & 1, bars, p);
            if (!ok) break;
            ptx::tc_fence_after();
            if (ptx::elect_one()) {
                output(i, buf, j > 0);
                if (j + 1 < u.steps[i]) scores(i, nbuf);
                else                    ptx::mma_commit(&bars->ofull[i]);
            }
            __syncwarp();
        }
        if (ok && ptx::elect_one()) {
            ptx::mma_commit(&bars->vempty[buf]);
            if (j + 1 < steps) ptx::mma_commit(&bars->kempty[nbuf]);
        }
        __syncwarp();
    }
    if (ptx::elect_one()) {                          // issued MMAs finish before TMEM is freed
        ptx::mma_commit(&bars->teardown);
        wait_drain(&bars->teardown, 0, p.c.status);
    }
    __syncwarp();
}

// ---------------------------------------------------------------- the rows
// One step of a row: its 128 products (tensor memory, `ts`) -> weights (fp16, over them), the running
// maximum m (log2) and sum l; O at `to` follows a new maximum.  In units of log2 a score is
// z = s f + a with f = qf s_k >= 0, a = log2 s_v per 16 tokens, so that a group's largest
// score is that of its largest product.  The products are read twice, 32 at a time with the next 32
// on the way, for the maximum and for the weights: a read takes some 80 cycles for all 128, and
// holding them leaves too few registers to keep the exponentials flowing.  EDGE: tokens at or past
// `left` are not seen.
template <bool EDGE>
__device__ __forceinline__ float chunk_top(const uint32_t (&s)[32], const GroupInfo* gi, int32_t left, float qf) {
    float top = -INFINITY;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        float g0 = -INFINITY, g1 = -INFINITY;
#pragma unroll
        for (int e = 0; e < 16; e += 4) {
            const float x[4] = {__uint_as_float(s[16 * h + e]), __uint_as_float(s[16 * h + e + 1]),
                                __uint_as_float(s[16 * h + e + 2]), __uint_as_float(s[16 * h + e + 3])};
            if (!EDGE) {
                g0 = fmaxf(fmaxf(g0, x[0]), x[1]);
                g1 = fmaxf(fmaxf(g1, x[2]), x[3]);
            } else {
#pragma unroll
                for (int y = 0; y < 4; ++y)
                    if (16 * h + e + y < left) g0 = fmaxf(g0, x[y]);
            }
        }
        g0 = fmaxf(g0, g1);
        const float2 q = *reinterpret_cast<const float2*>(&gi[h]);
        const float z = fmaf(g0, qf * q.x, q.y);
        top = fmaxf(top, EDGE && g0 == -INFINITY ? -INFINITY : z);
    }
    return top;
}
template <bool EDGE>
__device__ __forceinline__ void chunk_weights(const uint32_t (&s)[32], const GroupInfo* gi, int32_t left, float qf, float base,
                                              float& l, uint32_t (&w)[16]) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const float4 q = *reinterpret_cast<const float4*>(&gi[h]);
        const float2 f2 = make_float2(qf * q.x, qf * q.x), a2 = make_float2(q.y - base, q.y - base);
        float2 part[2] = {make_float2(0.0f, 0.0f), make_float2(0.0f, 0.0f)};
#pragma unroll
        for (int e = 0; e < 16; e += 2) {
            float2 z = fma2_rn(make_float2(__uint_as_float(s[16 * h + e]), __uint_as_float(s[16 * h + e + 1])), f2, a2);
            if (EDGE && 16 * h + e >= left) z.x = -INFINITY;
            if (EDGE && 16 * h + e + 1 >= left) z.y = -INFINITY;
            const float2 y = make_float2(ex2(z.x), ex2(z.y));
            part[(e >> 1) & 1] = add2_rn(part[(e >> 1) & 1], y);
            w[8 * h + e / 2] = pack_half2(y.x, y.y);
        }
        const float2 sum = add2_rn(part[0], part[1]);
        l = fmaf(sum.x + sum.y, q.z, l);
    }
}

template <int D, bool EDGE>
__device__ __forceinline__ void weights(const GroupInfo* gi, int32_t left, float qf, float& m, float& l, bool has_o,
                                        uint32_t ts, uint32_t to) {
    uint32_t s0[32], s1[32];
    ptx::tmem_ld_32x32b_x32(ts, s0);
    ptx::tmem_ld_wait();
    float top = -INFINITY;                                 // with P_SHIFT in it
#pragma unroll
    for (int c = 0; c < 4; c += 2) {
        ptx::tmem_ld_32x32b_x32(ts + 32 * (c + 1), s1);
        top = fmaxf(top, chunk_top<EDGE>(s0, gi + 2 * c, left - 32 * c, qf));
        ptx::tmem_ld_wait();
        ptx::tmem_ld_32x32b_x32(ts + 32 * ((c + 2) & 3), s0);      // the last: the first again
        top = fmaxf(top, chunk_top<EDGE>(s1, gi + 2 * c + 2, left - 32 * c - 32, qf));
        ptx::tmem_ld_wait();
    }
    const bool far = m == -INFINITY ? top > -INFINITY : top > m + (P_SHIFT + P_LAG);
    if (__any_sync(0xffffffffu, far)) {
        const float m_new = fmaxf(m, top - P_SHIFT);
        const float corr = m_new == -INFINITY ? 1.0f : ex2(m - m_new);
        m = m_new;
        l *= corr;
        if (has_o) {
#pragma unroll 1
            for (int c = 0; c < D / 16; ++c) {
                uint32_t o[16];
                ptx::tmem_ld_32x32b_x16(to + 16 * c, o);
                ptx::tmem_ld_wait();
#pragma unroll
                for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * corr);
                ptx::tmem_st_32x32b_x16(to + 16 * c, o);
            }
        }
    }
    const float base = m == -INFINITY ? 0.0f : m;
#pragma unroll
    for (int c = 0; c < 4; c += 2) {
        uint32_t w[16];
        ptx::tmem_ld_32x32b_x32(ts + 32 * (c + 1), s1);
        chunk_weights<EDGE>(s0, gi + 2 * c, left - 32 * c, qf, base, l, w);
        ptx::tmem_ld_wait();
        ptx::tmem_st_32x32b_x16(ts + 16 * c, w);           // over products that have been read
        if (c == 0) ptx::tmem_ld_32x32b_x32(ts + 64, s0);
        chunk_weights<EDGE>(s1, gi + 2 * c + 2, left - 32 * c - 32, qf, base, l, w);
        if (c == 0) ptx::tmem_ld_wait();
        ptx::tmem_st_32x32b_x16(ts + 16 * c + 16, w);
    }
}

// Warps 8-11 (i = 0) and 12-15 (i = 1): thread = row = TMEM lane.
template <int D>
__device__ __forceinline__ void rows(const AttnParams& p, const Unit& u, uint8_t* q16, const GroupInfo (*info)[T_GROUPS],
                                     uint32_t tmem, Bars* bars) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int i = (warp - 8) >> 2;
    const uint32_t quarter = warp & 3;
    const int32_t trow = quarter * 32 + lane;                       // row of the tile
    const int32_t row = u.row0 + i * T_ROWS + trow;
    const bool real = row < u.rows;
    const int32_t limit = real ? sees_upto(p, u.s, row) : 0x7fffffff;
    const int32_t least = __reduce_min_sync(0xffffffffu, limit);
    // ---- Q: divided by a power of two, as fp16, in 64-element blocks
    float qf;
    {
        const uint16_t* src = p.q + (int64_t)(u.s.first + (real ? row / p.group : 0)) * p.ldq +
                              (int64_t)(u.h * p.group + (real ? row % p.group : 0)) * D;
        uint32_t m2 = 0;
        for (int k = 0; k < D / 8; ++k) {
            const uint4 v = real ? ld_v4(src + 8 * k) : make_uint4(0, 0, 0, 0);
            m2 = max_bf16x2_bits(m2, max_bf16x2_bits(max_bf16x2_bits(abs_bf16x2(v.x), abs_bf16x2(v.y)),
                                                     max_bf16x2_bits(abs_bf16x2(v.z), abs_bf16x2(v.w))));
        }
        const int e = max(1, min((int)(hmax_pair(m2) >> 7), 253));
        // the sign of the softmax scale goes into Q, so that the largest product is the largest score
        const float inv = copysignf(__uint_as_float((uint32_t)(254 - e) << 23), p.scale2);
        qf = __uint_as_float((uint32_t)e << 23) * fabsf(p.scale2);
        for (int k = 0; k < D / 8; ++k) {
            const uint4 v = real ? ld_v4(src + 8 * k) : make_uint4(0, 0, 0, 0);
            *reinterpret_cast<uint4*>(q16 + i * tile_bytes<D>() + (k >> 3) * T_BLOCK + swizzled(trow, k & 7)) =
                make_uint4(pack_half2(bf16_lo(v.x) * inv, bf16_hi(v.x) * inv), pack_half2(bf16_lo(v.y) * inv, bf16_hi(v.y) * inv),
                           pack_half2(bf16_lo(v.z) * inv, bf16_hi(v.z) * inv), pack_half2(bf16_lo(v.w) * inv, bf16_hi(v.w) * inv));
        }
        ptx::fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(&bars->qfull);
    }
    const uint32_t lane_base = (quarter * 32) << 16;
    const uint32_t ts = tmem + lane_base + i * T_TOK, to = tmem + lane_base + 2 * T_TOK + i * D;
    float m = -INFINITY, l = 0.0f;
    for (int32_t j = 0; j < u.steps[i]; ++j) {
        if (!warp_wait(&bars->sfull[i], j & 1, bars, p)) return;
        ptx::tc_fence_after();
        const GroupInfo* gi = info[j & 3];
        const int32_t left = limit - j * T_TOK;
        if (least - j * T_TOK < T_TOK)                     // some row of the warp ends in this step
            weights<D, true>(gi, left, qf, m, l, j > 0, ts, to);
        else
            weights<D, false>(gi, left, qf, m, l, j > 0, ts, to);
        ptx::tmem_st_wait();
        ptx::tc_fence_before();
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(&bars->pfull[i]);
    }
    if (u.steps[i] == 0) return;
    if (!warp_wait(&bars->ofull[i], 0, bars, p)) return;
    ptx::tc_fence_after();
    const float inv = l > 0.0f ? __frcp_rn(l) : 0.0f;
    uint16_t* dst = real ? out_row(p, u.s, u.h, row, D) : nullptr;
#pragma unroll 1
    for (int c = 0; c < D / 32; ++c) {
        uint32_t o[32];
        ptx::tmem_ld_32x32b_x32(to + 32 * c, o);
        ptx::tmem_ld_wait();
        if (real) {
#pragma unroll
            for (int e = 0; e < 32; e += 8)
                *reinterpret_cast<uint4*>(dst + 32 * c + e) =
                    make_uint4(pack_bf16x2(__uint_as_float(o[e]) * inv, __uint_as_float(o[e + 1]) * inv),
                               pack_bf16x2(__uint_as_float(o[e + 2]) * inv, __uint_as_float(o[e + 3]) * inv),
                               pack_bf16x2(__uint_as_float(o[e + 4]) * inv, __uint_as_float(o[e + 5]) * inv),
                               pack_bf16x2(__uint_as_float(o[e + 6]) * inv, __uint_as_float(o[e + 7]) * inv));
        }
    }
}

template <int FMT, int D>
__global__ void __launch_bounds__(T_THREADS, 1) kv_prompt_attention_kernel(const __grid_constant__ AttnParams p) {
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    Bars* bars = reinterpret_cast<Bars*>(smem);
    GroupInfo (*info)[T_GROUPS] = reinterpret_cast<GroupInfo (*)[T_GROUPS]>(smem + 256);   // 4 steps
    uint8_t* q16 = smem + T_HEADER;
    uint8_t* k16 = q16 + 2 * tile_bytes<D>();
    uint8_t* v16 = k16 + 2 * tile_bytes<D>();
    const int warp = threadIdx.x >> 5;
    // of each sequence the CTAs with the most tokens to see (the last rows) come first; the sequences go side by side
    // whatever their lengths
    const int32_t bh = p.c.batch * p.c.kv_heads;
    const int32_t rt = p.row_tiles - 1 - (int32_t)(blockIdx.x / bh);
    Unit u;
    u.b = (int32_t)(blockIdx.x % bh) / p.c.kv_heads;
    u.h = (int32_t)(blockIdx.x % bh) % p.c.kv_heads;
    u.s = sequence_of(p.c, u.b, p.max_kv);
    if (!u.s.ok) {
        if (rt == 0 && threadIdx.x == 0) report_status(p.c.status, FP8_ERR_INVALID_ARG);
        return;
    }
    u.rows = u.s.n * p.group;
    u.row0 = rt * T_CTA_ROWS;
    if (u.row0 >= u.rows) return;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int32_t first = u.row0 + i * T_ROWS, last = min(first + T_ROWS, u.rows) - 1;
        u.steps[i] = first < u.rows ? max(1, (sees_upto(p, u.s, last) + T_TOK - 1) / T_TOK) : 0;
    }
    u.sees = sees_upto(p, u.s, min(u.row0 + T_CTA_ROWS, u.rows) - 1);
    if (threadIdx.x == 0) {
        for (int i = 0; i < 2; ++i) {
            ptx::mbar_init(&bars->kfull[i], 4);
            ptx::mbar_init(&bars->vfull[i], 4);
            ptx::mbar_init(&bars->kempty[i], 1);
            ptx::mbar_init(&bars->vempty[i], 1);
            ptx::mbar_init(&bars->sfull[i], 1);
            ptx::mbar_init(&bars->pfull[i], 4);
            ptx::mbar_init(&bars->ofull[i], 1);
        }
        ptx::mbar_init(&bars->qfull, 8);
        ptx::mbar_init(&bars->teardown, 1);
        bars->abort_flag = 0;
        ptx::fence_mbar_init();
    }
    if (warp == 1) {
        ptx::tmem_alloc(&bars->tmem_slot, 512);
        ptx::tmem_relinquish();
    }
    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
    const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(&bars->tmem_slot);
    // registers: 128 a thread at launch, 512 for the four warpgroups together; 56 + 120 + 2 * 168 = 512
    if (warp < 4) {
        ptx::regs_dec<56>();
        if (warp == 0) {
            // the same in all lanes, and known to be: the MMAs take their operands from uniform registers
            auto uniform = [](uint32_t x) { return __shfl_sync(0xffffffffu, x, 0); };
            issue<D>(p, u, uniform(ptx::smem_u32(q16)), uniform(ptx::smem_u32(k16)), uniform(ptx::smem_u32(v16)),
                     uniform(tmem), bars);
        }
    } else if (warp < 8) {
        ptx::regs_dec<120>();
        convert<FMT, D>(p, u, k16, v16, info, bars);
    } else {
        ptx::regs_inc<168>();
        rows<D>(p, u, q16, info, tmem, bars);
    }
    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
    if (warp == 1) ptx::tmem_dealloc(tmem, 512);
}

template <int FMT, int D>
cudaError_t launch_prompt(AttnParams p, cudaStream_t st) {
    static bool attr_done[kDeviceCacheSlots];   // the attribute is set per device
    const int ds = device_slot();
    if (ds < 0 || !attr_done[ds]) {
        const cudaError_t e = cudaFuncSetAttribute(kv_prompt_attention_kernel<FMT, D>,
                                                   cudaFuncAttributeMaxDynamicSharedMemorySize, (int)prompt_smem<D>());
        if (e != cudaSuccess) return e;
        if (ds >= 0) attr_done[ds] = true;
    }
    const int64_t rows = (int64_t)p.c.max_q * p.group;
    p.row_tiles = (int32_t)((rows + T_CTA_ROWS - 1) / T_CTA_ROWS);
    const int64_t ctas = prompt_ctas(p.c.batch, p.c.kv_heads, rows);
    if (ctas >= ((int64_t)1 << 31)) return cudaErrorInvalidConfiguration;
    kv_prompt_attention_kernel<FMT, D><<<(unsigned)ctas, T_THREADS, prompt_smem<D>(), st>>>(p);
    return cudaGetLastError();
}

}  // namespace

int64_t prompt_ctas(int32_t batch, int32_t kv_heads, int64_t rows) {
    return (int64_t)batch * kv_heads * ((rows + T_CTA_ROWS - 1) / T_CTA_ROWS);
}

cudaError_t launch_prompt_attention(const AttnParams& p, cudaStream_t st) {
    if (p.c.fmt == FP8_E4M3)
        return p.c.head_dim == 128 ? launch_prompt<FP8_E4M3, 128>(p, st) : launch_prompt<FP8_E4M3, 64>(p, st);
    return p.c.head_dim == 128 ? launch_prompt<FP8_E5M2, 128>(p, st) : launch_prompt<FP8_E5M2, 64>(p, st);
}

}  // namespace fp8b
