// norm.cu -- residual addition + root-mean-square norm + FP8 output (sm_100a).
//
//   h = x + r,  y = h / sqrt(mean(h^2) + eps) * w,  (q, s) = quantise(y)
//
// All in fp32 from the bf16 inputs; h, y and the codes are each rounded once from the fp32
// values.  The work is 2 B read (4 with a residual) and 1 B written (3 with h) per element
// and some ten instructions, so HBM bounds it: a row is read once, with every load of a
// thread issued before the first use, stays in registers through its two reductions (the
// sum of squares; the amax, over the row or a 128- or 32-element group of it), and is
// written once.  The division by the scale is the corrected reciprocal of quantize.cu.
// Measured: 16384 x 8192 with a residual, 1x128 scales (939 MB) 148 us in a burst = 6.3 TB/s, 151-168
// sustained (a plain copy of as many bytes, sustained: 151); 1 row of 8192 2.4 us; 1021 x 5152, MX32,
// 5.8 us.
#include "common.cuh"
#include "kernels.h"

namespace fp8b {

namespace {

constexpr int NVEC = 8;            // bf16 elements per 16-byte vector
constexpr int WARP_ROWS = 8;       // rows (warps) of a CTA in the warp-per-row kernel

struct NormParams {
    const uint16_t* x;
    const uint16_t* res;
    uint16_t* sum;
    const uint16_t* weight;
    uint8_t* q;
    void* scale;
    uint16_t* y;
    const float* amax_in;
    int32_t* status;
    int64_t rows, ldx, ldr, lds;
    int32_t cols, nvec, nscale;    // nscale: scales per row
    float eps, inv_cols;
};

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// Sum (max) over the group of threads that owns a row: a warp, or the CTA through `red`.
template <bool WARP>
__device__ __forceinline__ float group_sum(float v, float* red) {
    v = warp_sum(v);
    if (WARP) return v;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, nw = blockDim.x >> 5;
    if (lane == 0) red[warp] = v;
    __syncthreads();
    return warp_sum(lane < nw ? red[lane] : 0.0f);
}
template <bool WARP>
__device__ __forceinline__ uint32_t group_max(uint32_t v, uint32_t* red) {
    v = __reduce_max_sync(0xffffffffu, v);
    if (WARP) return v;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, nw = blockDim.x >> 5;
    if (lane == 0) red[warp] = v;
    __syncthreads();
    return __reduce_max_sync(0xffffffffu, lane < nw ? red[lane] : 0u);
}

__device__ __forceinline__ float2 unpack2(uint32_t w) { return make_float2(bf16_lo(w), bf16_hi(w)); }
__device__ __forceinline__ uint32_t word(const uint4& v, int i) { return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w; }
__device__ __forceinline__ uint4 pack8(const float2* f) {
    return make_uint4(pack_bf16x2(f[0].x, f[0].y), pack_bf16x2(f[1].x, f[1].y), pack_bf16x2(f[2].x, f[2].y),
                      pack_bf16x2(f[3].x, f[3].y));
}

// -y for 8 values -> 8 codes of y / s (r = RN(1/s), one Markstein step on -y, which keeps the sign of
// a zero, as in quantize.cu; a quotient that overflows, possible with a given amax only,
// saturates uncorrected).
template <int FMT, bool GUARD>
__device__ __forceinline__ uint2 encode8(const float2* ny, float s, float r) {
    uint32_t c[4];
    const float2 nr = make_float2(-r, -r), s2 = make_float2(s, s);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 q = mul2_rn(ny[i], nr);
        float2 t = fma2_rn(fma2_rn(q, s2, ny[i]), nr, q);
        if (GUARD) {
            if (!(fabsf(q.x) <= 3.402823466e38f)) t.x = q.x;
            if (!(fabsf(q.y) <= 3.402823466e38f)) t.y = q.y;
        }
        c[i] = cvt_pair<FMT>(t.x, t.y);
    }
    return make_uint2(c[0] | (c[1] << 16), c[2] | (c[3] << 16));
}

// max(|a|, |b|), NaN if either is.
__device__ __forceinline__ float max_abs_nan(float a, float b) {
    float d;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(fabsf(a)), "f"(fabsf(b)));
    return d;
}

// MODE: fp8_scaling_t.  VPT: 16-byte vectors of a row per thread.  WARP: a warp per row
// (rows of up to 32 VPT vectors), else the CTA (blockDim.x >= nvec / VPT).  ANY_EPS: for an eps that the plain
// forms of the root do not serve (see launch_mode).
template <int FMT, int MODE, int VPT, bool WARP, bool ANY_EPS>
__global__ void __launch_bounds__(WARP ? 32 * WARP_ROWS : 1024) rmsnorm_quantize_kernel(const NormParams p) {
    __shared__ float red_sum[2][32];
    __shared__ uint32_t red_max[32];
    const int64_t row = WARP ? (int64_t)blockIdx.x * WARP_ROWS + (threadIdx.x >> 5) : (int64_t)blockIdx.x;
    if (WARP && row >= p.rows) return;
    const int t = WARP ? (threadIdx.x & 31) : threadIdx.x;
    const int step = WARP ? 32 : blockDim.x;
    float2 h[VPT][NVEC / 2];
    uint4 wv[VPT];
    {
        uint4 xv[VPT], rv[VPT];
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
            const int k = t + j * step;
            xv[j] = make_uint4(0, 0, 0, 0);
            if (k < p.nvec) xv[j] = ld_v4_stream(p.x + row * p.ldx + k * NVEC);
        }
        if (p.res) {
#pragma unroll
            for (int j = 0; j < VPT; ++j) {
                const int k = t + j * step;
                rv[j] = make_uint4(0, 0, 0, 0);
                if (k < p.nvec) rv[j] = ld_v4_stream(p.res + row * p.ldr + k * NVEC);
            }
        }
        // the weight comes from L2, ahead of the reduction that it follows
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
            const int k = t + j * step;
            wv[j] = make_uint4(0x3F803F80u, 0x3F803F80u, 0x3F803F80u, 0x3F803F80u);
            if (p.weight && k < p.nvec) wv[j] = __ldg(reinterpret_cast<const uint4*>(p.weight + k * NVEC));
        }
#pragma unroll
        for (int j = 0; j < VPT; ++j)
#pragma unroll
            for (int i = 0; i < NVEC / 2; ++i) {
                h[j][i] = unpack2(word(xv[j], i));
                if (p.res) h[j][i] = add2_rn(h[j][i], unpack2(word(rv[j], i)));
            }
    }
    float2 ss2 = make_float2(0.0f, 0.0f);
#pragma unroll
    for (int j = 0; j < VPT; ++j)
#pragma unroll
        for (int i = 0; i < NVEC / 2; ++i) ss2 = fma2_rn(h[j][i], h[j][i], ss2);
    const float ss = group_sum<WARP>(ss2.x + ss2.y, red_sum[0]);
    if (p.sum) {
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
            const int k = t + j * step;
            if (k < p.nvec) st_v4_stream(p.sum + row * p.lds + k * NVEC, pack8(h[j]));
        }
    }
    // 1 / sqrt(mean + eps); squares that leave the fp32 range (|h| above 1e19) are summed again at 2^-80 of
    // their size, where eps is far below; with ANY_EPS also a sum that eps takes out of the range or
    // leaves near subnormals, at 2^60 then, and eps at the square.  The branch is the same for the whole row.
    float rstd;
    auto again = [&](float pre) {
        float s2 = 0.0f;
#pragma unroll
        for (int j = 0; j < VPT; ++j)
#pragma unroll
            for (int i = 0; i < NVEC / 2; ++i) {
                s2 = fmaf(h[j][i].x * pre, h[j][i].x * pre, s2);
                s2 = fmaf(h[j][i].y * pre, h[j][i].y * pre, s2);
            }
        s2 = group_sum<WARP>(s2, red_sum[1]) * p.inv_cols;
        // at 2^-80 the product may be subnormal, with 21 bits at least
        return pre * __frsqrt_rn(ANY_EPS ? fmaf(p.eps * pre, pre, s2) : s2);
    };
    const float down = 8.271806125530277e-25f, up = 1.152921504606847e18f;                     // 2^-80, 2^60
    if (!ANY_EPS) {
        if (ss <= 3.402823466e38f) rstd = __frsqrt_rn(fmaf(ss, p.inv_cols, p.eps));
        else                       rstd = again(down);
    } else {
        const float mean = fmaf(ss, p.inv_cols, p.eps);
        if (mean < 7.888609052210118e-31f)   rstd = again(up);                                  // 2^-100
        else if (!(mean <= 3.402823466e38f)) rstd = again(down);
        else                                 rstd = __frsqrt_rn(mean);
    }
    // h becomes -y
    float m[VPT];
    float top = 0.0f;
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
        m[j] = 0.0f;
#pragma unroll
        for (int i = 0; i < NVEC / 2; ++i) {
            h[j][i] = mul2_rn(mul2_rn(h[j][i], make_float2(-rstd, -rstd)), unpack2(word(wv[j], i)));
            m[j] = max_abs_nan(m[j], max_abs_nan(h[j][i].x, h[j][i].y));
        }
        top = max_abs_nan(top, m[j]);
    }
    const uint32_t all = __float_as_uint(top) & 0x7FFFFFFFu;     // patterns order like the values, NaN above
    float s = 1.0f, r = 1.0f;
    if (MODE == FP8_SCALE_ROW) {
        uint32_t a = group_max<WARP>(all, red_max);
        if (a >= 0x7F800000u) {
            if (t == 0) report_status(p.status, FP8_ERR_NONFINITE);
            a = 0x7F7FFFFFu;
        }
        s = scale_from_amax<FMT>(__uint_as_float(a));
        r = __frcp_rn(s);
        if (t == 0) static_cast<float*>(p.scale)[row] = s;
    } else if (MODE == FP8_SCALE_TENSOR) {
        if (all >= 0x7F800000u) report_status(p.status, FP8_ERR_NONFINITE);
        float a = *p.amax_in;
        if (!(a <= 3.402823466e38f)) {
            if (row == 0 && t == 0) report_status(p.status, FP8_ERR_NONFINITE);
            a = 3.402823466e38f;
        }
        s = scale_from_amax<FMT>(a);
        r = __frcp_rn(s);
        if (row == 0 && t == 0) static_cast<float*>(p.scale)[0] = s;
    }
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
        const int k = t + j * step;
        if (MODE == FP8_SCALE_BLOCK_1x128 || MODE == FP8_SCALE_MX32) {
            // a block is 16 (4) vectors, held by as many neighbouring lanes
            uint32_t a = __float_as_uint(m[j]) & 0x7FFFFFFFu;
#pragma unroll
            for (int o = MODE == FP8_SCALE_MX32 ? 2 : 8; o > 0; o >>= 1)
                a = max(a, __shfl_xor_sync(0xffffffffu, a, o));
            if (a >= 0x7F800000u) {
                if (k < p.nvec) report_status(p.status, FP8_ERR_NONFINITE);
                a = 0x7F7FFFFFu;
            }
            if (MODE == FP8_SCALE_MX32) {
                const int e = mx_exponent(a >> 16);      // the exponent is in the upper bits
                r = exp2i(-e);
                if ((k & 3) == 0 && k < p.nvec)
                    static_cast<uint8_t*>(p.scale)[row * p.nscale + (k >> 2)] = (uint8_t)(e + 127);
            } else {
                s = scale_from_amax<FMT>(__uint_as_float(a));
                r = __frcp_rn(s);
                if ((k & 15) == 0 && k < p.nvec) static_cast<float*>(p.scale)[row * p.nscale + (k >> 4)] = s;
            }
        }
        if (k >= p.nvec) continue;
        uint2 c;
        if (MODE == FP8_SCALE_MX32) {
            uint32_t w[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float2 q = mul2_rn(h[j][i], make_float2(-r, -r));
                w[i] = cvt_pair<FMT>(q.x, q.y);
            }
            c = make_uint2(w[0] | (w[1] << 16), w[2] | (w[3] << 16));
        } else {
            c = encode8<FMT, MODE == FP8_SCALE_TENSOR>(h[j], s, r);
        }
        *reinterpret_cast<uint2*>(p.q + row * p.cols + k * NVEC) = c;
        if (p.y) {
            uint4 y = pack8(h[j]);
            y.x ^= 0x80008000u;
            y.y ^= 0x80008000u;
            y.z ^= 0x80008000u;
            y.w ^= 0x80008000u;
            st_v4_stream(p.y + row * p.cols + k * NVEC, y);
        }
    }
}

template <int FMT, int MODE, int VPT, bool WARP, bool ANY_EPS = false>
cudaError_t launch_one(const NormParams& p, cudaStream_t st) {
    const int64_t grid = WARP ? (p.rows + WARP_ROWS - 1) / WARP_ROWS : p.rows;
    const int per = (p.nvec + VPT - 1) / VPT;
    const int threads = WARP ? 32 * WARP_ROWS : std::max(32, (per + 31) / 32 * 32);
    rmsnorm_quantize_kernel<FMT, MODE, VPT, WARP, ANY_EPS><<<(unsigned)grid, threads, 0, st>>>(p);
    return cudaGetLastError();
}

template <int FMT, int MODE>
cudaError_t launch_mode(const NormParams& p, cudaStream_t st) {
    // Below 2^-126 eps does not cover the rounding of subnormal squares, and above 2^88 it counts beside sums that
    // leave fp32 or takes them there.  These rows have an instance of their own: in the others its
    // branches would cost registers, and with them 5 to 10 % (1021 x 5152, MX32: 5.8 and 6.3 us).
    if (!(p.eps >= 1.1754943508e-38f && p.eps <= 3.0948500982e26f))
        return p.nvec <= 128 ? launch_one<FMT, MODE, 4, true, true>(p, st) : launch_one<FMT, MODE, 4, false, true>(p, st);
    if (p.nvec <= 32) return launch_one<FMT, MODE, 1, true>(p, st);
    if (p.nvec <= 64) return launch_one<FMT, MODE, 2, true>(p, st);
    if (p.nvec <= 128) return launch_one<FMT, MODE, 4, true>(p, st);
    // two vectors per thread for few rows, where a row's latency counts, and for rows of up to 2,048;
    // four otherwise, where fewer and longer-lived threads leave HBM busier (with 2 and with 4: 1 row of
    // 8192 2.4 and 2.7 us, 256 rows 3.9 and 4.1, 1021 x 5152 5.8 and 6.3, 16384 x 1088 24 and 29;
    // 4096 x 8192 46 and 38, 16384 x 8192 156 and 150)
    if (p.nvec <= 256 || (p.rows <= 1024 && p.nvec <= 2048)) return launch_one<FMT, MODE, 2, false>(p, st);
    return launch_one<FMT, MODE, 4, false>(p, st);     // nvec <= 4096: at most 1024 threads
}

template <int FMT>
cudaError_t launch_fmt(const NormParams& p, int32_t mode, cudaStream_t st) {
    switch (mode) {
    case FP8_SCALE_TENSOR: return launch_mode<FMT, FP8_SCALE_TENSOR>(p, st);
    case FP8_SCALE_ROW: return launch_mode<FMT, FP8_SCALE_ROW>(p, st);
    case FP8_SCALE_BLOCK_1x128: return launch_mode<FMT, FP8_SCALE_BLOCK_1x128>(p, st);
    default: return cudaErrorInvalidValue;
    }
}

// TENSOR with nothing to quantise still writes its scale.
template <int FMT>
__global__ void given_scale_kernel(const float* amax, float* scale, int32_t* status) {
    float a = *amax;
    if (!(a <= 3.402823466e38f)) {
        report_status(status, FP8_ERR_NONFINITE);
        a = 3.402823466e38f;
    }
    *scale = scale_from_amax<FMT>(a);
}

}  // namespace

cudaError_t launch_rmsnorm_quantize(const NormArgs& a, cudaStream_t st) {
    if (a.rows == 0 || a.cols == 0) {                    // TENSOR only: the caller fills the others
        if (a.fmt == FP8_E4M3) given_scale_kernel<FP8_E4M3><<<1, 1, 0, st>>>(a.amax_in, static_cast<float*>(a.scale), a.status);
        else                   given_scale_kernel<FP8_E5M2><<<1, 1, 0, st>>>(a.amax_in, static_cast<float*>(a.scale), a.status);
        return cudaGetLastError();
    }
    NormParams p{};
    p.x = a.x;
    p.res = a.res;
    p.sum = a.sum;
    p.weight = a.weight;
    p.q = a.q;
    p.scale = a.scale;
    p.y = a.y;
    p.amax_in = a.amax_in;
    p.status = a.status;
    p.rows = a.rows;
    p.ldx = a.ldx;
    p.ldr = a.ldr;
    p.lds = a.lds;
    p.cols = (int32_t)a.cols;
    p.nvec = (int32_t)(a.cols / NVEC);
    p.nscale = a.mode == FP8_SCALE_MX32 ? p.cols / 32 : (p.cols + 127) / 128;
    p.eps = a.eps;
    p.inv_cols = 1.0f / (float)a.cols;
    if (a.mode == FP8_SCALE_MX32) return launch_mode<FP8_E4M3, FP8_SCALE_MX32>(p, st);
    return a.fmt == FP8_E4M3 ? launch_fmt<FP8_E4M3>(p, a.mode, st) : launch_fmt<FP8_E5M2>(p, a.mode, st);
}

}  // namespace fp8b
