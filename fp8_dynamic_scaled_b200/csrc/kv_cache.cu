// kv_cache.cu -- quantises new tokens' K and V into the pages of an FP8 cache (sm_100a).
//
// Per page and KV head one scale s = 2^e, the least e with max(amax, 1e-12) <= F_max 2^e.  FP8
// codes are floating-point, so within its range a power-of-two scale costs no precision, and
// it makes growth of a page's scale harmless: the earlier codes move by a factor 2^-k, which
// is exact unless they become subnormal.  (With s = amax / F_max every growth would round all
// earlier codes of the page once more.)
//
// One group of threads per (page that the call touches, KV head, K or V): it reads the page's
// new tokens (in registers), reduces their amax, moves the earlier codes if the scale grew, and
// writes the codes.  2 B read and 1 B written per element: HBM bounds long prompts, latency a
// decode step.  A decode step's units hold one token (a 256-byte row at head_dim 128), for which
// a warp is enough; longer calls give a unit 256 threads, 8 vectors each at most.
#include "kv_common.cuh"

namespace fp8b {

namespace {

constexpr int APPEND_THREADS = 256;
constexpr int APPEND_VPT = 8;        // 128 tokens x 128 / 8 elements per vector / 256 threads
constexpr int DECODE_VPT = 4;        // per lane of the warp variant

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

template <int FMT, bool WARP>
__global__ void __launch_bounds__(APPEND_THREADS) kv_append_kernel(const __grid_constant__ AppendParams p) {
    constexpr int VPT = WARP ? DECODE_VPT : APPEND_VPT;
    constexpr int GROUP = WARP ? 32 : APPEND_THREADS;
    __shared__ uint32_t red[APPEND_THREADS / 32];
    const KvArgs& c = p.c;
    const int32_t unit = WARP ? (int32_t)blockIdx.y * (APPEND_THREADS / 32) + (threadIdx.x >> 5) : (int32_t)blockIdx.y;
    if (unit >= 2 * c.kv_heads) return;
    const int t = WARP ? (threadIdx.x & 31) : threadIdx.x;
    const int32_t head = unit >> 1, which = unit & 1;
    const int32_t b = (int32_t)(blockIdx.x / p.slots), slot = (int32_t)(blockIdx.x % p.slots);
    const Sequence s = sequence_of(c, b, (int64_t)1 << 30);
    if (!s.ok || s.n > s.kv_len) {
        if (t == 0 && slot == 0) report_status(c.status, FP8_ERR_INVALID_ARG);
        return;
    }
    if (s.n == 0) return;
    const int32_t P = c.page_size, D = c.head_dim;
    const int32_t start = s.kv_len - s.n;
    const int32_t index = start / P + slot;                          // entry of the page table
    const int32_t lo = max(start, index * P), hi = min(s.kv_len, (index + 1) * P);
    if (lo >= hi) return;
    const int32_t page = __ldg(c.table + (int64_t)b * c.table_stride + index);
    if (page < 0 || page >= c.num_pages) {
        if (t == 0) report_status(c.status, FP8_ERR_INVALID_ARG);
        return;
    }
    const int32_t held = lo - index * P;                             // earlier tokens of the page
    const int64_t at = (int64_t)page * c.kv_heads + head;
    uint8_t* codes = (which ? c.v : c.k) + at * P * D;
    float* scale = (which ? c.v_scale : c.k_scale) + at;
    const int32_t vec_row = D / 8, shift = D == 128 ? 4 : 3;
    const int32_t nvec = (hi - lo) * vec_row;
    const uint16_t* src = p.x[which] + (int64_t)(s.first + lo - start) * p.ld[which] + (int64_t)head * D;
    uint4 x[VPT];
    uint32_t m2 = 0;
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
        const int32_t k = t + j * GROUP;
        x[j] = make_uint4(0, 0, 0, 0);
        if (k < nvec) x[j] = ld_v4_stream(src + (int64_t)(k >> shift) * p.ld[which] + (k & (vec_row - 1)) * 8);
    }
#pragma unroll
    for (int j = 0; j < VPT; ++j)
        m2 = max_bf16x2_bits(m2, max_bf16x2_bits(max_bf16x2_bits(abs_bf16x2(x[j].x), abs_bf16x2(x[j].y)),
                                                 max_bf16x2_bits(abs_bf16x2(x[j].z), abs_bf16x2(x[j].w))));
    const float old = held > 0 ? *scale : 0.0f;
    uint32_t m = __reduce_max_sync(0xffffffffu, hmax_pair(m2));
    if (!WARP) {
        if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = m;
        __syncthreads();                                             // also: every thread has read `old`
        m = 0;
#pragma unroll
        for (int i = 0; i < APPEND_THREADS / 32; ++i) m = max(m, red[i]);
    } else {
        __syncwarp();
    }
    if (m >= 0x7F80u) {
        if (t == 0) report_status(c.status, FP8_ERR_NONFINITE);
        m = 0x7F7Fu;
    }
    const float now = fmaxf(old, page_scale<FMT>(fmaxf(bf16bits_to_float(m), amax_floor())));
    if (t == 0) *scale = now;
    const float inv = __frcp_rn(now);                                // exact: a power of two
    if (held > 0 && now != old) {
        const float f = __fmul_rn(old, inv);
        const int32_t n16 = held * D / 16;
        for (int32_t k = t; k < n16; k += GROUP) {
            uint4* w = reinterpret_cast<uint4*>(codes) + k;
            uint4 v = *w;
            v.x = rescale4<FMT>(v.x, f);
            v.y = rescale4<FMT>(v.y, f);
            v.z = rescale4<FMT>(v.z, f);
            v.w = rescale4<FMT>(v.w, f);
            *w = v;
        }
    }
    uint8_t* dst = codes + (int64_t)held * D;
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
        const int32_t k = t + j * GROUP;
        if (k >= nvec) continue;
        const uint32_t w[4] = {x[j].x, x[j].y, x[j].z, x[j].w};
        uint32_t o[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) o[i] = cvt_pair<FMT>(__fmul_rn(bf16_lo(w[i]), inv), __fmul_rn(bf16_hi(w[i]), inv));
        reinterpret_cast<uint2*>(dst)[k] = make_uint2(o[0] | (o[1] << 16), o[2] | (o[3] << 16));
    }
}

template <int FMT, bool WARP>
cudaError_t launch_append(const AppendParams& p, cudaStream_t st) {
    const int units = 2 * p.c.kv_heads;
    const dim3 grid((unsigned)((int64_t)p.c.batch * p.slots),
                    (unsigned)(WARP ? (units + APPEND_THREADS / 32 - 1) / (APPEND_THREADS / 32) : units));
    kv_append_kernel<FMT, WARP><<<grid, APPEND_THREADS, 0, st>>>(p);
    return cudaGetLastError();
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
    const bool warp = std::min<int64_t>(longest, c.page_size) * (c.head_dim / 8) <= 32 * DECODE_VPT;
    if (c.fmt == FP8_E4M3) return warp ? launch_append<FP8_E4M3, true>(p, st) : launch_append<FP8_E4M3, false>(p, st);
    return warp ? launch_append<FP8_E5M2, true>(p, st) : launch_append<FP8_E5M2, false>(p, st);
}

}  // namespace fp8b
