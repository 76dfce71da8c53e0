// attention.cu -- causal attention of bf16 queries over the paged FP8 cache (sm_100a).
//
//   out[t, h] = sum_j p_j v_j,  p = softmax_j(scale q[t, h] . k_j),  j up to t's own position
//
// One pass over the cached tokens with a running maximum and sum.  The heads that share a KV
// head are rows of one tile (rows = query tokens x group, 8 or 16 of them), so that a page is read
// once for all of them.  Operands of the products are fp16: FP8 codes are fp16 values (no rounding);
// a query row is first divided by a power of two so that its largest element is in [1, 2); the
// weights are scaled to 2^8 .. 2^15 for the largest, so that fp16 keeps 11 bits of a weight
// down to 2^-22 of it.  Scores, softmax statistics and sums are fp32.
//
// The page's scales: with z = scale q . code_k * s_k in units of log2, the running maximum M is
// taken over z + log2 s_v, and the weight is w = 2^(z + log2 s_v - M + 8): sum w code_v is then
// sum p v without a product per page, whatever the spread of s_v among pages, and the sum of
// the softmax is sum w / s_v.  M may lag behind the true maximum by 2^7, which fp16 has room
// for: the sums are moved to a new M only when a score passes that, a rare event after the
// first tiles.
//
// The kernel here is for few rows, where the codes' bytes bound it: 2 D of them per cached token
// and KV head, read once.  Measured: 64 sequences of up to 8192 tokens, 64 / 8 heads of 128, 135 us
// = 5.7 TB/s of codes (0.88 of a plain copy's rate); 2 of 100,001 tokens, 32 / 4 heads, 44 us, of
// which some 12 are latency (lengths, pages, first codes, joining); 1 of 333 tokens 12.7 us.  An
// earlier form with a CTA per (sequence, KV head, split of 512 tokens or more), each warp loading its
// codes straight into registers, took 236, 100 and 10 us: 8 warps per SM could not keep enough
// bytes in flight, and 16-row products left half of each instruction empty.
#include "attention_common.cuh"

namespace fp8b {

namespace {

constexpr int A_TOK = 32;             // tokens of a work tile: one ring stage, one warp
constexpr int A_HEADER = 1024;        // barriers, the CTA's place in the work
constexpr int A_MAX_STAGES = 24;
constexpr int A_SMEM = 227 * 1024;

// 8 or 16 rows per tile (NQ = 1, 2).  With 8 the accumulators leave room for 16 warps per SM (128
// registers), with 16 for 12 (168 registers).
template <int D, int NQ>
struct Shape {
    static constexpr int ROWS = 8 * NQ;
    static constexpr int WARPS = NQ == 1 ? 10 : 8;                  // consumers
    static constexpr int PRODUCERS = NQ == 1 ? 4 : 2;               // warps that fill the ring
    static constexpr int THREADS = 32 * (WARPS + PRODUCERS + 1);    // and the joining warp
    static constexpr int LD = D + 4;                                // floats per row of a warp's part
    static constexpr int PART_BYTES = WARPS * ROWS * LD * 4;
    static constexpr int ML_BYTES = WARPS * ROWS * 8;
    static constexpr int STAGE = 2 * A_TOK * D;
    static constexpr int FIT = (A_SMEM - 1024 - A_HEADER - PART_BYTES - ML_BYTES - A_MAX_STAGES * 32) / STAGE;
    // Every stage belongs to one producer and one consumer.  A warp then sees each phase of its
    // stages' barriers in turn; a consumer that shared its stages with others could ask for a
    // phase while the barrier is two phases behind, which a parity cannot tell from done.
    static constexpr int TURN = NQ == 1 ? 20 : 8;
    static constexpr int STAGES = (FIT < A_MAX_STAGES ? FIT : A_MAX_STAGES) / TURN * TURN;
    static_assert(TURN % WARPS == 0 && TURN % PRODUCERS == 0 && STAGES > 0, "stages have one owner on each side");
};

__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// The 8 x 8 block of 16-bit values that a warp holds in fragment layout, transposed.
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}

// ---------------------------------------------------------------- the work list
// A unit is (sequence, KV head, row tile of 8 or 16 rows = query tokens x group); its work tiles
// are 32 cached tokens each, up to the last token that one of its rows sees (one tile, without
// tokens, when they see none).  The tiles of all units in a row are cut into equal ranges, one
// for each CTA, whatever the lengths: a CTA works through the end of one unit, whole units
// and the beginning of another.
__device__ __forceinline__ int32_t rows_of(const AttnParams& p, const Sequence& s) { return s.ok ? s.n * p.group : 0; }

// Tokens that row tile rt's last row sees.
template <int ROWS>
__device__ __forceinline__ int32_t tile_sees(const AttnParams& p, const Sequence& s, int32_t rt) {
    const int32_t last = min((rt + 1) * ROWS, s.n * p.group) - 1;
    return max(0, s.kv_len - s.n + last / p.group + 1);
}
__device__ __forceinline__ int32_t tiles_of(int32_t sees) { return max(1, (sees + A_TOK - 1) / A_TOK); }

// Work tiles of one KV head of a sequence.
template <int ROWS>
__device__ __forceinline__ int64_t head_tiles(const AttnParams& p, const Sequence& s) {
    const int32_t rts = (rows_of(p, s) + ROWS - 1) / ROWS;
    int64_t n = 0;
    for (int32_t rt = 0; rt < rts; ++rt) n += tiles_of(tile_sees<ROWS>(p, s, rt));
    return n;
}

// This CTA's range of the work and where it begins: the whole CTA calls it.
struct Range {
    int64_t lo;
    int32_t n;                        // tiles of the range
    int64_t each;                     // tiles of every CTA, one more for the first `extra`
    int32_t extra;
    // The CTA that has tile x of the whole list.
    __device__ __forceinline__ int32_t cta_of(int64_t x) const {
        const int64_t longer = extra * (each + 1);
        return (int32_t)(x < longer ? x / (each + 1) : extra + (x - longer) / each);
    }
};
struct Start {
    int64_t inside;                   // tiles of sequence b before the range
    int32_t b;
};

template <class S>
__device__ Range find_range(const AttnParams& p, Start* start, int64_t* sums /* [32] */) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, nw = S::THREADS / 32;
    const int32_t per = (p.c.batch + S::THREADS - 1) / S::THREADS;
    const int32_t b0 = (int32_t)threadIdx.x * per, b1 = min(p.c.batch, b0 + per);
    int64_t mine = 0;
    for (int32_t b = b0; b < b1; ++b) {
        const Sequence s = sequence_of(p.c, b, p.max_kv);
        if (!s.ok && blockIdx.x == 0) report_status(p.c.status, FP8_ERR_INVALID_ARG);
        mine += head_tiles<S::ROWS>(p, s) * p.c.kv_heads;
    }
    int64_t incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t v = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += v;
    }
    if (lane == 31) sums[warp] = incl;
    __syncthreads();
    Range r;
    int64_t before = 0, total = 0;
    for (int w = 0; w < nw; ++w) {
        if (w < warp) before += sums[w];
        total += sums[w];
    }
    // a CTA's warps share its tiles: fewer CTAs when there is not one tile for each warp
    const int32_t ctas = (int32_t)max((int64_t)1, min((int64_t)gridDim.x, (total + S::WARPS - 1) / S::WARPS));
    const int32_t i = (int32_t)blockIdx.x;
    r.each = total / ctas;
    r.extra = (int32_t)(total - r.each * ctas);
    r.lo = i < ctas ? r.each * i + min(i, r.extra) : total;
    r.n = i < ctas ? (int32_t)r.each + (i < r.extra ? 1 : 0) : 0;
    const int64_t first = before + incl - mine;
    if (r.lo >= first && r.lo < first + mine) {
        int64_t at = first;
        for (int32_t b = b0; b < b1; ++b) {
            const int64_t n = head_tiles<S::ROWS>(p, sequence_of(p.c, b, p.max_kv)) * p.c.kv_heads;
            if (r.lo < at + n) {
                start->b = b;
                start->inside = r.lo - at;
                break;
            }
            at += n;
        }
    }
    __syncthreads();
    return r;
}

// The unit at hand, walking through a range.
template <int ROWS>
struct Cursor {
    int32_t b, h, rt, rts;
    Sequence s;
    int32_t sees, tiles;              // of the unit

    __device__ __forceinline__ void unit(const AttnParams& p) {
        sees = tile_sees<ROWS>(p, s, rt);
        tiles = tiles_of(sees);
    }
    __device__ __forceinline__ void sequence(const AttnParams& p, int32_t b0) {
        b = b0;
        s = sequence_of(p.c, b, p.max_kv);
        rts = (rows_of(p, s) + ROWS - 1) / ROWS;
        h = rt = 0;
    }
    __device__ __forceinline__ void next(const AttnParams& p) {
        if (++rt == rts) {
            rt = 0;
            if (++h == p.c.kv_heads) {
                do { sequence(p, b + 1); } while (rts == 0 && b + 1 < p.c.batch);
            }
        }
        unit(p);
    }
    // The unit of the range's first tile; returns the tiles of that unit before the range.
    __device__ __forceinline__ int32_t open(const AttnParams& p, const Start& st) {
        sequence(p, st.b);
        int64_t inside = st.inside;
        const int64_t per_head = head_tiles<ROWS>(p, s);
        h = (int32_t)(inside / per_head);
        inside -= h * per_head;
        unit(p);
        while (inside >= tiles) {
            inside -= tiles;
            ++rt;
            unit(p);
        }
        return (int32_t)inside;
    }
};

// ---------------------------------------------------------------- the ring
// One stage: 32 tokens of K, then of V, D bytes each, as TMA wrote them (128-byte rows with the
// 128-byte swizzle, or 64-byte rows with the 64-byte one), and the tile's numbers.
struct __align__(16) StageInfo {
    float ks[2], lv[2], iv[2];        // per 16 tokens: s_k, log2 s_v + P_SHIFT, 1 / s_v
    int32_t valid[2];                 // tokens of the 16 that are there
};

template <int D>
__device__ __forceinline__ uint32_t stage_chunk(uint32_t row, uint32_t chunk) {   // byte offset of 16 bytes
    return D == 128 ? row * 128 + ((chunk ^ (row & 7)) << 4) : row * 64 + ((chunk ^ ((row >> 1) & 3)) << 4);
}

struct Ring {
    uint8_t* data;
    StageInfo* info;
    uint64_t *full, *empty;
    volatile int32_t* abort_flag;
};

// The range's tile g sits in stage g % STAGES; it is fetched by producer g % PRODUCERS and used
// by consumer g % WARPS.  (One producer warp could not keep up: a tile costs it about 700
// cycles, and at HBM's rate an SM takes one every 350.)
template <int D, class S>
__device__ __forceinline__ void produce(const AttnParams& p, const CUtensorMap& tk, const CUtensorMap& tv,
                                        const Range& range, const Start& st, const Ring& ring, int32_t who) {
    const int lane = threadIdx.x & 31;
    const int32_t P = p.c.page_size;
    Cursor<S::ROWS> c;
    int32_t off = c.open(p, st);
    IssuedLoads loads;
    int32_t stage = who, phase = 0;
    bool ok = true;
    int32_t mine = who;                                    // this warp's next tile of the range
    for (int32_t n = 0; n < range.n && ok;) {
        const int32_t count = min(c.tiles - off, range.n - n);
        while (mine < n + count && ok) {
            // lane i looks up the page and the scales of tile mine + i PRODUCERS
            const int32_t k = off + (mine - n) + lane * S::PRODUCERS;
            int32_t row[2] = {-1, -1};
            StageInfo si;
#pragma unroll
            for (int g = 0; g < 2; ++g) {
                si.ks[g] = si.iv[g] = 1.0f;
                si.lv[g] = P_SHIFT;
                si.valid[g] = 0;
                const int32_t tok = k * A_TOK + 16 * g;
                if (k >= off + count || tok >= c.sees) continue;
                const int32_t page = __ldg(p.c.table + (int64_t)c.b * p.c.table_stride + tok / P);
                if (page < 0 || page >= p.c.num_pages) {
                    report_status(p.c.status, FP8_ERR_INVALID_ARG);
                    continue;
                }
                const int64_t at = (int64_t)page * p.c.kv_heads + c.h;
                row[g] = (int32_t)(at * P + tok % P);
                si.ks[g] = __ldg(p.c.k_scale + at);
                const float vs = __ldg(p.c.v_scale + at);
                if (!v_scale_ok(vs)) report_status(p.c.status, FP8_ERR_INVALID_ARG);
                si.lv[g] = __log2f(vs) + P_SHIFT;
                si.iv[g] = __frcp_rn(vs);
                si.valid[g] = min(16, c.sees - tok);
            }
            for (int32_t j = 0; j < 32 && mine < n + count; ++j, mine += S::PRODUCERS) {
                if (ok) ok = wait_limited(&ring.empty[stage], (phase & 1) ^ 1, ring.abort_flag, p.c.status, p.wait_ns);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) break;
                if (lane == j) ring.info[stage] = si;
                const int32_t row0 = __shfl_sync(0xffffffffu, row[0], j), row1 = __shfl_sync(0xffffffffu, row[1], j);
                __syncwarp();
                if (lane == 0) {
                    uint8_t* dst = ring.data + stage * S::STAGE;
                    // a copy of 32 rows covers both halves (they are in one page)
                    const int32_t copies = p.box == A_TOK ? (row0 >= 0 ? 1 : 0) : (row0 >= 0) + (row1 >= 0);
                    ptx::mbar_arrive_expect_tx(&ring.full[stage], (uint32_t)(2 * copies * p.box * D));
                    if (row0 >= 0) {
                        ptx::tma_load_2d(dst, &tk, &ring.full[stage], 0, row0);
                        ptx::tma_load_2d(dst + A_TOK * D, &tv, &ring.full[stage], 0, row0);
                    }
                    if (row1 >= 0 && p.box != A_TOK) {
                        ptx::tma_load_2d(dst + 16 * D, &tk, &ring.full[stage], 0, row1);
                        ptx::tma_load_2d(dst + (A_TOK + 16) * D, &tv, &ring.full[stage], 0, row1);
                    }
                }
                loads.note((uint32_t)stage, (uint32_t)phase);
                __syncwarp();
                stage += S::PRODUCERS;
                if (stage >= S::STAGES) stage -= S::STAGES, ++phase;
            }
        }
        n += count;
        off = 0;
        if (n < range.n) c.next(p);
    }
    __syncwarp();
    if (lane == 0) loads.drain(ring.full, p.c.status);     // every copy has landed before the CTA may exit
}

// ---------------------------------------------------------------- the consumers
// Fragment layouts (c = lane % 4, r = lane / 4; mma m16n8k16).  The cached tokens (for the scores)
// and the head's elements (for the output) are the instruction's 16 rows, the queries its 8
// columns: grouped heads of 8 rows then waste no half of an instruction.
//   scores[token, q] = K Q^T: the reduction index is permuted so that a lane's operands are 16
//     contiguous bytes of a token's K row (chunk 2c + h at D = 128, c at 64: each phase of
//     eight lanes then reads all banks once).
//   out[d, q] += V^T W: m-tile j holds d = (D / 8) row + 2j, + 1 (rows r, r + 8), so that a lane's
//     operands are D / 8 contiguous bytes of a V row.  W [token, q] leaves the scores'
//     accumulator layout through an 8 x 8 transposition.
template <int FMT, int D, int NQ>
struct Consumer {
    static constexpr int KK = D / 16;          // k-steps of the scores
    static constexpr int MT = D / 16;          // m-tiles of the output
    static constexpr int CH = D / 64;          // 16-byte chunks of a K row per lane
    uint32_t qb[NQ][KK][2];
    float qf[NQ][2];                           // of queries 8 nq + 2c, + 1
    int32_t limit[NQ][2];                      // tokens the query sees (0: no such row)
    int32_t least;                             // tokens the tile's first row sees
    float o[NQ][MT][4], m[NQ][2], l[NQ][2];

    __device__ __forceinline__ void open(const AttnParams& p, const Cursor<8 * NQ>& u) {
        const int lane = threadIdx.x & 31, c = lane & 3, r = lane >> 2;
        const int32_t rows = u.s.n * p.group, row0 = u.rt * 8 * NQ;
        least = max(0, u.s.kv_len - u.s.n + row0 / p.group + 1);
#pragma unroll
        for (int i = 0; i < NQ; ++i) {
            const int32_t row = row0 + r + 8 * i;
            const bool real = row < rows;
            const int32_t tok = real ? row / p.group : 0;
            const uint16_t* src = p.q + (int64_t)(u.s.first + tok) * p.ldq +
                                  (int64_t)(u.h * p.group + (real ? row % p.group : 0)) * D + 16 * CH * c;
            uint4 v[CH][2];
            uint32_t m2 = 0;
#pragma unroll
            for (int h = 0; h < CH; ++h)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    v[h][e] = real ? ld_v4(src + 16 * h + 8 * e) : make_uint4(0, 0, 0, 0);
                    m2 = max_bf16x2_bits(m2, max_bf16x2_bits(max_bf16x2_bits(abs_bf16x2(v[h][e].x), abs_bf16x2(v[h][e].y)),
                                                             max_bf16x2_bits(abs_bf16x2(v[h][e].z), abs_bf16x2(v[h][e].w))));
                }
            uint32_t top = hmax_pair(m2);
            top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
            top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
            const int e = max(1, min((int)(top >> 7), 253));                // biased exponent of the row's largest
            const float inv = __uint_as_float((uint32_t)(254 - e) << 23);   // 2^(127 - e)
            const float f = __uint_as_float((uint32_t)e << 23) * p.scale2;
            const int32_t lim = real ? max(0, u.s.kv_len - u.s.n + tok + 1) : 0;
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                qf[i][x] = __shfl_sync(0xffffffffu, f, 4 * (2 * c + x));
                limit[i][x] = __shfl_sync(0xffffffffu, lim, 4 * (2 * c + x));
                m[i][x] = -INFINITY;
                l[i][x] = 0.0f;
            }
#pragma unroll
            for (int h = 0; h < CH; ++h)
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const uint32_t w0 = k < 2 ? (k == 0 ? v[h][0].x : v[h][0].z) : (k == 2 ? v[h][1].x : v[h][1].z);
                    const uint32_t w1 = k < 2 ? (k == 0 ? v[h][0].y : v[h][0].w) : (k == 2 ? v[h][1].y : v[h][1].w);
                    qb[i][4 * h + k][0] = pack_half2(bf16_lo(w0) * inv, bf16_hi(w0) * inv);
                    qb[i][4 * h + k][1] = pack_half2(bf16_lo(w1) * inv, bf16_hi(w1) * inv);
                }
#pragma unroll
            for (int j = 0; j < MT; ++j)
#pragma unroll
                for (int x = 0; x < 4; ++x) o[i][j][x] = 0.0f;
        }
    }

    // One work tile: tokens tok0 .. tok0 + 31 in `st`.
    __device__ __forceinline__ void tile(const uint8_t* st, const StageInfo& si, int32_t tok0) {
        const int lane = threadIdx.x & 31, c = lane & 3, r = lane >> 2;
        // s[i][g][x + 2y]: token 16 g + r + 8 y, query 8 i + 2c + x
        float s[NQ][2][4];
#pragma unroll
        for (int i = 0; i < NQ; ++i)
#pragma unroll
            for (int g = 0; g < 2; ++g)
#pragma unroll
                for (int x = 0; x < 4; ++x) s[i][g][x] = 0.0f;
#pragma unroll
        for (int h = 0; h < CH; ++h) {
            uint4 v[2][2];
#pragma unroll
            for (int g = 0; g < 2; ++g)
#pragma unroll
                for (int y = 0; y < 2; ++y)
                    v[g][y] = *reinterpret_cast<const uint4*>(st + stage_chunk<D>(16 * g + 8 * y + r, CH * c + h));
#pragma unroll
            for (int k = 0; k < 4; ++k)
#pragma unroll
                for (int g = 0; g < 2; ++g) {
                    const uint32_t w0 = k == 0 ? v[g][0].x : k == 1 ? v[g][0].y : k == 2 ? v[g][0].z : v[g][0].w;
                    const uint32_t w1 = k == 0 ? v[g][1].x : k == 1 ? v[g][1].y : k == 2 ? v[g][1].z : v[g][1].w;
                    uint32_t a[4];
                    half2x2_of<FMT>(w0, a[0], a[2]);
                    half2x2_of<FMT>(w1, a[1], a[3]);
#pragma unroll
                    for (int i = 0; i < NQ; ++i) mma16816(s[i][g], a, qb[i][4 * h + k][0], qb[i][4 * h + k][1]);
                }
        }
        const float4 f0 = *reinterpret_cast<const float4*>(&si);        // ks[2], lv[2]
        const int4 f1 = *(reinterpret_cast<const int4*>(&si) + 1);      // iv[2], valid[2]
        const float ks[2] = {f0.x, f0.y}, lv[2] = {f0.z, f0.w};
        const float iv[2] = {__int_as_float(f1.x), __int_as_float(f1.y)};
        const int32_t valid[2] = {f1.z, f1.w};
        const bool edge = tok0 + A_TOK > least || valid[0] < 16 || valid[1] < 16;
        bool move = false;
        float top[NQ][2];
#pragma unroll
        for (int i = 0; i < NQ; ++i)
#pragma unroll
            for (int x = 0; x < 2; ++x) {
#pragma unroll
                for (int g = 0; g < 2; ++g) {
                    const float f = qf[i][x] * ks[g];
#pragma unroll
                    for (int y = 0; y < 2; ++y) s[i][g][x + 2 * y] = fmaf(s[i][g][x + 2 * y], f, lv[g]);
                }
            }
        if (edge) {
#pragma unroll
            for (int i = 0; i < NQ; ++i)
#pragma unroll
                for (int x = 0; x < 2; ++x)
#pragma unroll
                    for (int g = 0; g < 2; ++g)
#pragma unroll
                        for (int y = 0; y < 2; ++y)
                            if (tok0 + 16 * g + r + 8 * y >= limit[i][x] || r + 8 * y >= valid[g])
                                s[i][g][x + 2 * y] = -INFINITY;
        }
#pragma unroll
        for (int i = 0; i < NQ; ++i)
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                top[i][x] = fmaxf(fmaxf(s[i][0][x], s[i][0][x + 2]), fmaxf(s[i][1][x], s[i][1][x + 2])) - P_SHIFT;
                move |= top[i][x] > m[i][x] + P_LAG;
            }
        if (__any_sync(0xffffffffu, move)) {
#pragma unroll
            for (int i = 0; i < NQ; ++i)
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    float t = top[i][x];
#pragma unroll
                    for (int b = 4; b < 32; b <<= 1) t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, b));
                    t = fmaxf(t, m[i][x]);
                    const float corr = t == -INFINITY ? 1.0f : ex2(m[i][x] - t);
                    m[i][x] = t;
                    l[i][x] *= corr;
#pragma unroll
                    for (int j = 0; j < MT; ++j) {
                        o[i][j][x] *= corr;
                        o[i][j][x + 2] *= corr;
                    }
                }
        }
        uint32_t wb[NQ][2][2];                   // W as the B operand: [query][16 tokens][8 of them]
#pragma unroll
        for (int i = 0; i < NQ; ++i) {
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                const float base = m[i][x] == -INFINITY ? 0.0f : m[i][x];
#pragma unroll
                for (int g = 0; g < 2; ++g) {
#pragma unroll
                    for (int y = 0; y < 2; ++y) s[i][g][x + 2 * y] = ex2(s[i][g][x + 2 * y] - base);
                    l[i][x] = fmaf(s[i][g][x] + s[i][g][x + 2], iv[g], l[i][x]);
                }
            }
#pragma unroll
            for (int g = 0; g < 2; ++g)
#pragma unroll
                for (int y = 0; y < 2; ++y)
                    wb[i][g][y] = transpose8x8(pack_half2(s[i][g][2 * y], s[i][g][2 * y + 1]));
        }
        const uint8_t* sv = st + A_TOK * D;
        constexpr int NW = D / 32;               // words of V per lane and token
#pragma unroll
        for (int g = 0; g < 2; ++g) {
            uint32_t w[4][NW];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int tok = 2 * c + (i & 1) + 8 * (i >> 1);
                if (D == 128) {
                    const uint4 v = *reinterpret_cast<const uint4*>(sv + stage_chunk<D>(16 * g + tok, r));
                    w[i][0] = v.x; w[i][1] = v.y; w[i][NW - 2] = v.z; w[i][NW - 1] = v.w;
                } else {
                    const uint2 v = *reinterpret_cast<const uint2*>(sv + stage_chunk<D>(16 * g + tok, r >> 1) + 8 * (r & 1));
                    w[i][0] = v.x; w[i][1] = v.y;
                }
                // slots past the last token may hold anything: they count as zeros
                if (edge && tok >= valid[g]) {
#pragma unroll
                    for (int q = 0; q < NW; ++q) w[i][q] = 0;
                }
            }
#pragma unroll
            for (int q = 0; q < NW; ++q) {
                uint32_t a0[4], a1[4];           // m-tiles 2q and 2q + 1: d = .. + 4q, 4q + 1 and 4q + 2, 4q + 3
                half2x2_of<FMT>(__byte_perm(w[0][q], w[1][q], 0x5140), a0[0], a0[1]);
                half2x2_of<FMT>(__byte_perm(w[0][q], w[1][q], 0x7362), a1[0], a1[1]);
                half2x2_of<FMT>(__byte_perm(w[2][q], w[3][q], 0x5140), a0[2], a0[3]);
                half2x2_of<FMT>(__byte_perm(w[2][q], w[3][q], 0x7362), a1[2], a1[3]);
#pragma unroll
                for (int i = 0; i < NQ; ++i) {
                    mma16816(o[i][2 * q], a0, wb[i][g][0], wb[i][g][1]);
                    mma16816(o[i][2 * q + 1], a1, wb[i][g][0], wb[i][g][1]);
                }
            }
        }
    }

    // This warp's part of a unit, into shared memory.
    template <class S>
    __device__ __forceinline__ void put(float* part /* [ROWS][LD] */, float2* ml /* [ROWS] */) {
        const int lane = threadIdx.x & 31, c = lane & 3, r = lane >> 2;
#pragma unroll
        for (int i = 0; i < NQ; ++i)
#pragma unroll
            for (int x = 0; x < 2; ++x) {
#pragma unroll
                for (int b = 4; b < 32; b <<= 1) l[i][x] += __shfl_xor_sync(0xffffffffu, l[i][x], b);
                const int row = 8 * i + 2 * c + x;
                if (r == 0) ml[row] = make_float2(m[i][x], l[i][x]);
                float4* dst = reinterpret_cast<float4*>(part + row * S::LD + (D / 8) * r);
#pragma unroll
                for (int j = 0; j < MT; j += 2)
                    dst[j / 2] = make_float4(o[i][j][x], o[i][j][x + 2], o[i][j + 1][x], o[i][j + 1][x + 2]);
            }
    }
};

// The joining warp: sums the consumers' parts of each unit, and writes the output (a unit whose
// tiles are all in this range) or the CTA's part of it.
template <int D, class S>
__device__ __forceinline__ void join_parts(const AttnParams& p, const Range& range, const Start& st, const float* part,
                                           const float2* ml, uint64_t* jfull, uint64_t* jfree,
                                           volatile int32_t* abort_flag) {
    const int lane = threadIdx.x & 31;
    Cursor<S::ROWS> u;
    int32_t off = u.open(p, st);
    uint32_t seg = 0;
    int4 goes_on = make_int4(-1, 0, 0, 0);
    for (int32_t n = 0; n < range.n; ++seg) {
        const int32_t count = min(u.tiles - off, range.n - n);
        bool ok = wait_limited(jfull, seg & 1u, abort_flag, p.c.status, p.wait_ns);
        if (!__all_sync(0xffffffffu, ok)) break;
        const bool whole = count == u.tiles;
        const int32_t slot = 2 * (int32_t)blockIdx.x + (n == 0 ? 0 : 1);
        const int32_t rows = min(S::ROWS, u.s.n * p.group - u.rt * S::ROWS);
        for (int32_t row = 0; row < rows; ++row) {
            // lanes hold the warps' maxima and sums
            const float2 a = lane < S::WARPS ? ml[lane * S::ROWS + row] : make_float2(-INFINITY, 0.0f);
            float top = a.x;
#pragma unroll
            for (int b = 16; b > 0; b >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, b));
            const float f = top == -INFINITY ? 0.0f : ex2(a.x - top);
            float l = a.y * f;
#pragma unroll
            for (int b = 16; b > 0; b >>= 1) l += __shfl_xor_sync(0xffffffffu, l, b);
            constexpr int V = D / 32;
            float v[V];
#pragma unroll
            for (int e = 0; e < V; ++e) v[e] = 0.0f;
#pragma unroll
            for (int w = 0; w < S::WARPS; ++w) {
                const float g = __shfl_sync(0xffffffffu, f, w);
                const float* src = part + (w * S::ROWS + row) * S::LD + V * lane;
                if (V == 4) {
                    const float4 x = *reinterpret_cast<const float4*>(src);
                    v[0] = fmaf(x.x, g, v[0]); v[1] = fmaf(x.y, g, v[1]);
                    v[V - 2] = fmaf(x.z, g, v[V - 2]); v[V - 1] = fmaf(x.w, g, v[V - 1]);
                } else {
                    const float2 x = *reinterpret_cast<const float2*>(src);
                    v[0] = fmaf(x.x, g, v[0]); v[1] = fmaf(x.y, g, v[1]);
                }
            }
            if (whole) {
                const float inv = l > 0.0f ? __frcp_rn(l) : 0.0f;
                uint32_t* dst = reinterpret_cast<uint32_t*>(out_row(p, u.s, u.h, u.rt * S::ROWS + row, D)) + V / 2 * lane;
#pragma unroll
                for (int e = 0; e < V / 2; ++e) dst[e] = pack_bf16x2(v[2 * e] * inv, v[2 * e + 1] * inv);
            } else {
                float* dst = p.part_o + ((int64_t)slot * 16 + row) * D + V * lane;
#pragma unroll
                for (int e = 0; e < V; ++e) dst[e] = v[e];
                if (lane == 0) p.part_ml[(int64_t)slot * 16 + row] = make_float2(top, l);
            }
        }
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(jfree);
        n += count;
        if (n >= range.n && !whole && off == 0) {          // begins here, ends in a later CTA
            const int64_t last = range.lo + n - count + u.tiles - 1;
            goes_on = make_int4(u.b, u.h * p.row_tiles + u.rt, slot, range.cta_of(last));
        }
        off = 0;
        if (n < range.n) u.next(p);
    }
    if (lane == 0) p.joins[blockIdx.x] = goes_on;
}

template <int FMT, int D, int NQ>
__global__ void __launch_bounds__(Shape<D, NQ>::THREADS, 1)
kv_attention_kernel(const __grid_constant__ CUtensorMap tk, const __grid_constant__ CUtensorMap tv,
                    const __grid_constant__ AttnParams p) {
    using S = Shape<D, NQ>;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    Ring ring;
    ring.full = reinterpret_cast<uint64_t*>(smem);
    ring.empty = ring.full + A_MAX_STAGES;
    uint64_t* jfull = ring.empty + A_MAX_STAGES;
    uint64_t* jfree = jfull + 1;
    ring.abort_flag = reinterpret_cast<volatile int32_t*>(jfree + 1);
    Start* start = reinterpret_cast<Start*>(smem + 512);
    int64_t* sums = reinterpret_cast<int64_t*>(smem + 640);
    ring.data = smem + A_HEADER;
    float* part = reinterpret_cast<float*>(ring.data + S::STAGES * S::STAGE);
    float2* ml = reinterpret_cast<float2*>(reinterpret_cast<uint8_t*>(part) + S::PART_BYTES);
    ring.info = reinterpret_cast<StageInfo*>(reinterpret_cast<uint8_t*>(ml) + S::ML_BYTES);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    pdl_launch_dependents();                  // the joining kernel waits for this grid itself
    if (threadIdx.x == 0) {
        for (int i = 0; i < S::STAGES; ++i) {
            ptx::mbar_init(&ring.full[i], 1);
            ptx::mbar_init(&ring.empty[i], 1);
        }
        ptx::mbar_init(jfull, S::WARPS);
        ptx::mbar_init(jfree, 1);
        *ring.abort_flag = 0;
        ptx::fence_mbar_init();
        if (p.c.num_pages > 0) {              // else there are no maps (and no tokens)
            ptx::prefetch_tmap(&tk);
            ptx::prefetch_tmap(&tv);
        }
    }
    const Range range = find_range<S>(p, start, sums);       // syncs
    if (range.n == 0) {
        if (threadIdx.x == 0) p.joins[blockIdx.x] = make_int4(-1, 0, 0, 0);
        return;
    }
    if (warp >= S::WARPS) {
        if (warp == S::WARPS + S::PRODUCERS)
            join_parts<D, S>(p, range, *start, part, ml, jfull, jfree, ring.abort_flag);
        else
            produce<D, S>(p, tk, tv, range, *start, ring, warp - S::WARPS);
        return;
    }
    Cursor<S::ROWS> u;
    int32_t off = u.open(p, *start);
    Consumer<FMT, D, NQ> w;
    int32_t mine = warp;                      // this warp's next tile of the range
    int32_t stage = warp, phase = 0;
    while (stage >= S::STAGES) stage -= S::STAGES, ++phase;
    uint32_t seg = 0;
    bool ok = true;
    for (int32_t n = 0; n < range.n && ok; ++seg) {
        const int32_t count = min(u.tiles - off, range.n - n);
        w.open(p, u);
        while (mine < n + count) {
            // the lanes agree on a wait's outcome: the tile's shuffles need all of them
            ok = wait_limited(&ring.full[stage], phase & 1, ring.abort_flag, p.c.status, p.wait_ns);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
            w.tile(ring.data + stage * S::STAGE, ring.info[stage], (off + mine - n) * A_TOK);
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive(&ring.empty[stage]);
            mine += S::WARPS;
            stage += S::WARPS;
            while (stage >= S::STAGES) stage -= S::STAGES, ++phase;
        }
        // the parts' buffer is free once the unit before has been joined
        if (ok && seg > 0) ok = wait_limited(jfree, (seg - 1) & 1u, ring.abort_flag, p.c.status, p.wait_ns);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        w.template put<S>(part + warp * S::ROWS * S::LD, ml + warp * S::ROWS);
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(jfull);
        n += count;
        off = 0;
        if (n < range.n) u.next(p);
    }
}

// ---------------------------------------------------------------- the joining kernel
// A unit that several CTAs shared: its parts are slot j.z of the CTA where it begins and slot 0
// of each CTA up to the last.  A CTA joins 4 rows, J_GROUPS groups of threads per row
// taking every J_GROUPS-th part each.  (2 contexts of 100,000 tokens, 18 parts per unit, the whole
// call: 45.6 us with 4 groups whose threads each went over all maxima, 44.0 this way; a row per CTA with 16
// groups 43.3, but 13.0 us instead of 12.3 for one short sequence.)
constexpr int J_ROWS = 4, J_GROUPS = 8;

template <int D>
__global__ void __launch_bounds__(J_ROWS * J_GROUPS * D / 8)
kv_attention_join_kernel(const __grid_constant__ AttnParams p, int32_t tile_rows) {
    __shared__ float so[J_ROWS][J_GROUPS][D];
    __shared__ float sl[J_ROWS][J_GROUPS];
    pdl_wait();
    const int4 j = p.joins[blockIdx.x];
    if (j.x < 0) return;
    const Sequence s = sequence_of(p.c, j.x, p.max_kv);
    const int32_t h = j.y / p.row_tiles, rt = j.y % p.row_tiles;
    const int32_t parts = j.w - (int32_t)blockIdx.x + 1;
    constexpr int VEC = D / 8;
    // a warp's threads are of one row
    const int32_t d = (threadIdx.x % VEC) * 8, grp = threadIdx.x / VEC % J_GROUPS, lane = threadIdx.x & 31;
    const int32_t lrow = threadIdx.x / (VEC * J_GROUPS), row = blockIdx.y * J_ROWS + lrow;
    const bool real = rt * tile_rows + row < s.n * p.group;
    auto slot = [&](int32_t i) { return (int64_t)(i == 0 ? j.z : 2 * ((int32_t)blockIdx.x + i)) * 16 + row; };
    float m = -INFINITY;
    for (int32_t i = lane; real && i < parts; i += 32) m = fmaxf(m, p.part_ml[slot(i)].x);
#pragma unroll
    for (int b = 16; b > 0; b >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, b));
    float l = 0.0f, v[8] = {};
    if (m != -INFINITY) {
#pragma unroll 2
        for (int32_t i = grp; i < parts; i += J_GROUPS) {
            const int64_t at = slot(i);
            const float2 ml = p.part_ml[at];
            const float f = ex2(ml.x - m);
            l = fmaf(ml.y, f, l);
            const float4* src = reinterpret_cast<const float4*>(p.part_o + at * D + d);
            const float4 a = src[0], b = src[1];
            v[0] = fmaf(a.x, f, v[0]); v[1] = fmaf(a.y, f, v[1]); v[2] = fmaf(a.z, f, v[2]); v[3] = fmaf(a.w, f, v[3]);
            v[4] = fmaf(b.x, f, v[4]); v[5] = fmaf(b.y, f, v[5]); v[6] = fmaf(b.z, f, v[6]); v[7] = fmaf(b.w, f, v[7]);
        }
    }
    *reinterpret_cast<float4*>(&so[lrow][grp][d]) = make_float4(v[0], v[1], v[2], v[3]);
    *reinterpret_cast<float4*>(&so[lrow][grp][d + 4]) = make_float4(v[4], v[5], v[6], v[7]);
    if (d == 0) sl[lrow][grp] = l;
    __syncthreads();
    const int32_t e = 2 * (threadIdx.x % (VEC * J_GROUPS));          // two elements per thread
    if (e >= D || !real) return;
    float sum = 0.0f;
    float2 o = make_float2(0.0f, 0.0f);
#pragma unroll
    for (int g = 0; g < J_GROUPS; ++g) {
        sum += sl[lrow][g];
        const float2 x = *reinterpret_cast<const float2*>(&so[lrow][g][e]);
        o.x += x.x;
        o.y += x.y;
    }
    const float inv = sum > 0.0f ? __frcp_rn(sum) : 0.0f;
    *reinterpret_cast<uint32_t*>(out_row(p, s, h, rt * tile_rows + row, D) + e) = pack_bf16x2(o.x * inv, o.y * inv);
}

// ---------------------------------------------------------------- host side
template <int FMT, int D, int NQ>
cudaError_t launch_attention(AttnParams p, cudaStream_t st) {
    using S = Shape<D, NQ>;
    const int grid = num_sms();
    p.row_tiles = (int32_t)(((int64_t)p.c.max_q * p.group + S::ROWS - 1) / S::ROWS);
    const uint64_t rows = (uint64_t)p.c.num_pages * p.c.kv_heads * p.c.page_size;
    if (rows >= ((uint64_t)1 << 31)) return cudaErrorInvalidValue;    // beyond any GPU's memory
    p.box = std::min(p.c.page_size, A_TOK);
    CUtensorMap tk, tv;
    const CUtensorMapSwizzle sw = D == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B;
    memset(&tk, 0, sizeof(tk));
    memset(&tv, 0, sizeof(tv));
    if (rows > 0 && (!make_map_2d(&tk, CU_TENSOR_MAP_DATA_TYPE_UINT8, p.c.k, D, rows, D, D, p.box, sw) ||
                     !make_map_2d(&tv, CU_TENSOR_MAP_DATA_TYPE_UINT8, p.c.v, D, rows, D, D, p.box, sw)))
        return cudaErrorInvalidValue;
    static bool attr_done[kDeviceCacheSlots];   // the attribute is set per device
    const int ds = device_slot();
    if (ds < 0 || !attr_done[ds]) {
        const cudaError_t e = cudaFuncSetAttribute(kv_attention_kernel<FMT, D, NQ>,
                                                   cudaFuncAttributeMaxDynamicSharedMemorySize, A_SMEM);
        if (e != cudaSuccess) return e;
        if (ds >= 0) attr_done[ds] = true;
    }
    kv_attention_kernel<FMT, D, NQ><<<grid, S::THREADS, A_SMEM, st>>>(tk, tv, p);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid, S::ROWS / J_ROWS);
    cfg.blockDim = dim3(J_ROWS * J_GROUPS * D / 8);
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, kv_attention_join_kernel<D>, p, (int32_t)S::ROWS);
    return e != cudaSuccess ? e : cudaGetLastError();
}

// Whether the prompt kernel's tiles of 128 rows serve a call better than this file's of 16, by what both
// take (measured at D = 128 with sequences of one length, and used for D = 64 and ragged calls too): here 0.27 us
// per SM and work tile of 16 rows x 32 tokens, over all SMs, after 14 us; there 2.1 us per step of 128 tokens
// after 7 us, one CTA per SM, whose SMs are not shared among splits of a sequence.  E.g. 8 KV heads, 8 heads
// each, 4,096 cached tokens: 64 new tokens of 1 sequence 85 us here and 92 there, 128 new tokens 147 and 92; of
// 8 sequences 4 new tokens 51 and 76, 16 new tokens 141 and 79.  It is off by up to 1.3 near its border (64
// sequences of 512 tokens, 4 new ones: 85 us chosen, 65 possible), and it is one choice for the whole call, by
// the bounds of its longest sequence: 63 single tokens beside one chunk of 2048, all of 4,096 cached tokens,
// take 843 us, apart 98 and 274.
bool wide_tiles(const AttnParams& p) {
    const int64_t rows = (int64_t)p.c.max_q * p.group, units = (int64_t)p.c.batch * p.c.kv_heads;
    const double sms = num_sms();
    const double tiles = (double)units * (double)((rows + 15) / 16) * (double)((p.max_kv + A_TOK - 1) / A_TOK);
    const int64_t waves = (prompt_ctas(p.c.batch, p.c.kv_heads, rows) + (int64_t)sms - 1) / (int64_t)sms;
    return (double)waves * (7.0 + 2.1 * (double)((p.max_kv + 127) / 128)) < 14.0 + 0.27 * tiles / sms;
}

// 8 rows per tile where they hold all of a sequence's, else 16, or the prompt kernel's wide tiles.
template <int FMT, int D>
cudaError_t launch_rows(const AttnParams& p, cudaStream_t st) {
    if ((int64_t)p.c.max_q * p.group <= 8) return launch_attention<FMT, D, 1>(p, st);
    if (wide_tiles(p)) return launch_prompt_attention(p, st);
    return launch_attention<FMT, D, 2>(p, st);
}

}  // namespace

// The workspace: [2 grid][16][D] floats, the joins, then [2 grid][16] pairs.
size_t attention_workspace(int32_t head_dim) {
    return (size_t)num_sms() * (2 * 16 * (size_t)(head_dim + 2) * sizeof(float) + sizeof(int4));
}

cudaError_t launch_kv_attention(const AttnArgs& a, cudaStream_t st) {
    AttnParams p{};
    p.c = a.c;
    p.c.max_q = (int32_t)std::min<int64_t>(a.c.max_q, a.c.tokens);     // a loose bound sizes nothing
    p.q = a.q;
    p.out = a.out;
    p.ldq = a.ldq;
    p.ldo = a.ldo;
    p.max_kv = a.max_kv;
    p.q_heads = a.q_heads;
    p.group = a.q_heads / a.c.kv_heads;
    p.scale2 = a.softmax_scale * LOG2E;
    p.wait_ns = wait_limit_ns();
    const int64_t slots = 2 * (int64_t)num_sms();
    p.part_o = static_cast<float*>(a.workspace);
    p.joins = reinterpret_cast<int4*>(p.part_o + slots * 16 * a.c.head_dim);
    p.part_ml = reinterpret_cast<float2*>(p.joins + slots / 2);
    if (a.c.fmt == FP8_E4M3)
        return a.c.head_dim == 128 ? launch_rows<FP8_E4M3, 128>(p, st) : launch_rows<FP8_E4M3, 64>(p, st);
    return a.c.head_dim == 128 ? launch_rows<FP8_E5M2, 128>(p, st) : launch_rows<FP8_E5M2, 64>(p, st);
}

}  // namespace fp8b
