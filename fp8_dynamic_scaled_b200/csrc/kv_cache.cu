// kv_cache.cu -- quantises new tokens' K and V into the pages of an FP8 cache (sm_100a).
//
// Per page and KV head one scale s = 2^e, the least e with max(amax, 1e-12) <= F_max 2^e.  FP8
// codes are floating-point, so within its range a power-of-two scale costs no precision, and
// it makes growth of a page's scale harmless: the earlier codes move by a factor 2^-k, which
// is exact unless they become subnormal.  (With s = amax / F_max every growth would round all
// earlier codes of the page once more.)
//
// One group of threads per (page that the call touches, KV head): it reads the page's new K and V
// (in registers, 4 vectors of each per thread), reduces their amax, moves the earlier codes if a
// scale grew, and writes the codes.  2 B read and 1 B written per element: HBM bounds long
// prompts, latency a decode step.  A group is as large as its tokens need, from a warp (one token
// at head_dim 128 is 256 bytes) to 512 threads (a page of 128 tokens); K and V go together so
// that one lookup of the page (three dependent loads) is paid for twice the data.  7 prompts of
// up to 4096 tokens, 8 heads of 128, pages of 32: 59 us with 256 threads for each of K and V
// (three CTAs per SM), 21 us this way (5.1 TB/s; the ALU pipe is 72 % busy).
#include "kv_common.cuh"

namespace fp8b {

namespace {

constexpr int APPEND_VPT = 4;        // vectors of K (and of V) per thread

struct AppendParams {
    KvArgs c;
    const uint16_t* x[2];            // K, V
    int64_t ld[2];
    int32_t slots;                   // pages a sequence's tokens can touch
};

// The least power of two s with amax <= F_max s; F_max = 1.75 * 2^8 (E4M3), 1.75 * 2^15 (E5M2).
// amax is finite and at least 1e-12.
template <int FMT>
__device__ __forceinline__ float page_scale(float amax) {
    const uint32_t bits = __float_as_uint(amax);
    const int up = (bits & 0x7FFFFFu) > 0x600000u ? 1 : 0;          // mantissa above 1.75
    const int e = (int)(bits >> 23) - (FMT == FP8_E4M3 ? 8 : 15) + up;
    return __uint_as_float((uint32_t)e << 23);                      // e >= 72 for amax >= 1e-12
}

// 4 codes times a factor, rounded back to codes.
template <int FMT>
__device__ __forceinline__ uint32_t rescale4(uint32_t w, float f) {
    const float2 a = decode_pair<FMT>(w & 0xFFFFu), b = decode_pair<FMT>(w >> 16);
    return cvt_pair<FMT>(__fmul_rn(a.x, f), __fmul_rn(a.y, f)) |
           (cvt_pair<FMT>(__fmul_rn(b.x, f), __fmul_rn(b.y, f)) << 16);
}

// A page's scale for the call's tokens (|bf16| pattern m) over what it held (old, 0 for nothing).
template <int FMT>
__device__ __forceinline__ float scale_for(uint32_t m, float old) {
    return fmaxf(old, page_scale<FMT>(fmaxf(bf16bits_to_float(min(m, 0x7F7Fu)), amax_floor())));
}

template <int FMT, int GROUP>
__global__ void __launch_bounds__(GROUP > 256 ? GROUP : 256) kv_append_kernel(const __grid_constant__ AppendParams p) {
    constexpr int THREADS = GROUP > 256 ? GROUP : 256;
    constexpr int WARPS = GROUP / 32;               // of a group
    __shared__ uint2 red[THREADS / 32];
    const KvArgs& c = p.c;
    const int t = threadIdx.x % GROUP;
    const int32_t head = (int32_t)blockIdx.y * (THREADS / GROUP) + (int32_t)threadIdx.x / GROUP;
    const int32_t b = (int32_t)(blockIdx.x / p.slots), slot = (int32_t)(blockIdx.x % p.slots);
    const Sequence s = sequence_of(c, b, (int64_t)1 << 30);
    const int32_t P = c.page_size, D = c.head_dim;
    const int32_t start = s.kv_len - s.n;
    const int32_t index = (start >> (31 - __clz(P))) + slot;         // entry of the page table: P is a power of two
    const int32_t lo = max(start, index * P), hi = min(s.kv_len, (index + 1) * P);
    // the groups of a CTA go on together to the barrier, those without work among them
    bool work = head < c.kv_heads;
    if (!s.ok || start < 0) {
        if (work && head == 0 && t == 0 && slot == 0) report_status(c.status, FP8_ERR_INVALID_ARG);
        work = false;
    }
    if (lo >= hi) work = false;
    int32_t page = -1;
    if (work) {
        page = __ldg(c.table + (int64_t)b * c.table_stride + index);
        if (page < 0 || page >= c.num_pages) {
            if (t == 0) report_status(c.status, FP8_ERR_INVALID_ARG);
            work = false;
        }
    }
    const int32_t held = lo - index * P;                             // earlier tokens of the page
    const int64_t at = (int64_t)page * c.kv_heads + head;
    const int32_t vec_row = D / 8, shift = D == 128 ? 4 : 3;
    const int32_t nvec = work ? (hi - lo) * vec_row : 0;
    uint4 x[2][APPEND_VPT];
    uint32_t m[2] = {0, 0};
#pragma unroll
    for (int w = 0; w < 2; ++w) {
        const uint16_t* src = p.x[w] + (int64_t)(s.first + lo - start) * p.ld[w] + (int64_t)head * D;
#pragma unroll
        for (int j = 0; j < APPEND_VPT; ++j) {
            const int32_t k = t + j * GROUP;
            x[w][j] = make_uint4(0, 0, 0, 0);
            if (k < nvec) x[w][j] = ld_v4_stream(src + (int64_t)(k >> shift) * p.ld[w] + (k & (vec_row - 1)) * 8);
        }
    }
    float old[2] = {0.0f, 0.0f};
    if (work && held > 0) {
        old[0] = c.k_scale[at];
        old[1] = c.v_scale[at];
    }
#pragma unroll
    for (int w = 0; w < 2; ++w) {
        uint32_t m2 = 0;                                             // sign bits meaningless, NaN stays
#pragma unroll
        for (int j = 0; j < APPEND_VPT; ++j)
            m2 = bmax_abs_bf16x2(m2, bmax_abs_bf16x2(bmax_abs_bf16x2(x[w][j].x, x[w][j].y),
                                                     bmax_abs_bf16x2(x[w][j].z, x[w][j].w)));
        m[w] = __reduce_max_sync(0xffffffffu, hmax_pair(abs_bf16x2(m2)));
    }
    if (GROUP > 32) {
        if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = make_uint2(m[0], m[1]);
        __syncthreads();                                             // also: every thread has read `old`
#pragma unroll
        for (int i = 0; i < WARPS; ++i) {
            const uint2 r = red[threadIdx.x / GROUP * WARPS + i];
            m[0] = max(m[0], r.x);
            m[1] = max(m[1], r.y);
        }
    } else {
        __syncwarp();
    }
    if (!work) return;
    if (t == 0 && max(m[0], m[1]) >= 0x7F80u) report_status(c.status, FP8_ERR_NONFINITE);
#pragma unroll
    for (int w = 0; w < 2; ++w) {
        uint8_t* codes = (w ? c.v : c.k) + at * P * D;
        const float now = scale_for<FMT>(m[w], old[w]);
        const float inv = __frcp_rn(now);                            // exact: a power of two
        if (t == 0) (w ? c.v_scale : c.k_scale)[at] = now;
        if (held > 0 && now != old[w]) {
            const float f = __fmul_rn(old[w], inv);
            const int32_t n16 = held * D / 16;
            for (int32_t k = t; k < n16; k += GROUP) {
                uint4* q = reinterpret_cast<uint4*>(codes) + k;
                uint4 v = *q;
                v.x = rescale4<FMT>(v.x, f);
                v.y = rescale4<FMT>(v.y, f);
                v.z = rescale4<FMT>(v.z, f);
                v.w = rescale4<FMT>(v.w, f);
                *q = v;
            }
        }
        uint2* dst = reinterpret_cast<uint2*>(codes + (int64_t)held * D);
#pragma unroll
        for (int j = 0; j < APPEND_VPT; ++j) {
            const int32_t k = t + j * GROUP;
            if (k >= nvec) continue;
            const uint32_t q[4] = {x[w][j].x, x[w][j].y, x[w][j].z, x[w][j].w};
            uint32_t o[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float2 y = mul2_rn(make_float2(bf16_lo(q[i]), bf16_hi(q[i])), make_float2(inv, inv));
                o[i] = cvt_pair<FMT>(y.x, y.y);
            }
            dst[k] = make_uint2(o[0] | (o[1] << 16), o[2] | (o[3] << 16));
        }
    }
}

template <int FMT, int GROUP>
cudaError_t launch_append(const AppendParams& p, cudaStream_t st) {
    const int threads = GROUP > 256 ? GROUP : 256, heads = threads / GROUP;
    const dim3 grid((unsigned)((int64_t)p.c.batch * p.slots), (unsigned)((p.c.kv_heads + heads - 1) / heads));
    kv_append_kernel<FMT, GROUP><<<grid, threads, 0, st>>>(p);
    return cudaGetLastError();
}

// The smallest group whose threads hold a unit's vectors.
template <int FMT>
cudaError_t launch_append_fmt(const AppendParams& p, int64_t nvec, cudaStream_t st) {
    if (nvec <= 32 * APPEND_VPT) return launch_append<FMT, 32>(p, st);
    if (nvec <= 64 * APPEND_VPT) return launch_append<FMT, 64>(p, st);
    if (nvec <= 128 * APPEND_VPT) return launch_append<FMT, 128>(p, st);
    if (nvec <= 256 * APPEND_VPT) return launch_append<FMT, 256>(p, st);
    return launch_append<FMT, 512>(p, st);          // 128 tokens of 128 elements: 2048 vectors
}

}  // namespace

cudaError_t launch_kv_append(const KvArgs& c, const uint16_t* k, int64_t ldk, const uint16_t* v, int64_t ldv,
                             cudaStream_t st) {
    AppendParams p{};
    p.c = c;
    p.x[0] = k;
    p.x[1] = v;
    p.ld[0] = ldk;
    p.ld[1] = ldv;
    const int64_t longest = std::min<int64_t>(c.max_q, c.tokens);
    p.c.max_q = (int32_t)longest;
    p.slots = (int32_t)((longest + c.page_size - 2) / c.page_size + 1);
    if ((int64_t)p.slots * c.batch >= ((int64_t)1 << 31)) return cudaErrorInvalidConfiguration;
    const int64_t nvec = std::min<int64_t>(longest, c.page_size) * (c.head_dim / 8);
    return c.fmt == FP8_E4M3 ? launch_append_fmt<FP8_E4M3>(p, nvec, st) : launch_append_fmt<FP8_E5M2>(p, nvec, st);
}

}  // namespace fp8b
