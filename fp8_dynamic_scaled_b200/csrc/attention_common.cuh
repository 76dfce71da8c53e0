// attention_common.cuh -- what the kernels of fp8_kv_attention share: parameters, the decode of
// FP8 codes into fp16 pairs, and the constants of the scaled softmax weights (attention.cu
// states the mathematics).
#pragma once

#include "gemm_common.cuh"
#include "kv_common.cuh"

namespace fp8b {

constexpr float LOG2E = 1.4426950408889634f;
constexpr float P_SHIFT = 8.0f;        // the largest weight is 2^8 ..
constexpr float P_LAG = 7.0f;          // .. to 2^15 (fp16 ends at 2^16)

struct AttnParams {
    KvArgs c;
    const uint16_t* q;
    uint16_t* out;
    int64_t ldq, ldo, max_kv;
    int32_t q_heads, group;
    int32_t row_tiles;                // most row tiles of a (sequence, KV head)
    int32_t box;                      // page rows of one copy: min(page_size, A_TOK)
    float scale2;                     // softmax_scale * log2(e)
    float* part_o;                    // [2 grid][16][D]: a CTA's first and last part of a unit
    float2* part_ml;                  // [2 grid][16]: maximum (log2), sum
    int4* joins;                      // [grid]: the unit that begins in CTA i and goes on in the next
    uint64_t wait_ns;
};

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// The range of the V scales, 2^-56 to 2^24 (reported otherwise).  A weight w is 0 below 2^-126, while w / s_v counts
// in the softmax's sum whatever s_v is; and a part of the sum is dropped when its maximum is that far
// below another's.  With scales at most 2^80 apart what is lost is 2^-39 of the sum per token.
__device__ __forceinline__ bool v_scale_ok(float vs) { return vs >= 1.3877787807814457e-17f && vs <= 16777216.0f; }
// Four codes -> two pairs of fp16 values, exactly.
template <int FMT>
__device__ __forceinline__ void half2x2_of(uint32_t codes, uint32_t& lo, uint32_t& hi) {
    if (FMT == FP8_E4M3)
        asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, a;\n\t"
            "cvt.rn.f16x2.e4m3x2 %1, b;\n\t}" : "=r"(lo), "=r"(hi) : "r"(codes));
    else
        asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.rn.f16x2.e5m2x2 %0, a;\n\t"
            "cvt.rn.f16x2.e5m2x2 %1, b;\n\t}" : "=r"(lo), "=r"(hi) : "r"(codes));
}
__device__ __forceinline__ uint32_t pack_half2(float a, float b) {
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
}
// wait_bounded, but under a short limit (the failure-path tests) no test suspends the thread: these
// kernels' waits are short, and a test that suspends outlasts them.
__device__ __forceinline__ bool wait_limited(uint64_t* bar, uint32_t parity, volatile int32_t* abort_flag, int32_t* status,
                                             uint64_t limit_ns) {
    if (limit_ns >= 1000000ull) return wait_bounded(bar, parity, abort_flag, status, limit_ns);
    const uint64_t t0 = ptx::globaltimer();
    while (!ptx::mbar_test_wait(bar, parity)) {
        if (*abort_flag) return false;
        if (ptx::globaltimer() - t0 > limit_ns) {
            *abort_flag = 1;
            report_status(status, FP8_ERR_TIMEOUT);
            return false;
        }
    }
    return true;
}
__device__ __forceinline__ uint16_t* out_row(const AttnParams& p, const Sequence& s, int32_t h, int32_t row, int32_t D) {
    return p.out + (int64_t)(s.first + row / p.group) * p.ldo + (int64_t)(h * p.group + row % p.group) * D;
}

// attention_prompt.cu: rows of many query tokens on the tensor cores' wide tiles.
cudaError_t launch_prompt_attention(const AttnParams& p, cudaStream_t st);
int64_t prompt_ctas(int32_t batch, int32_t kv_heads, int64_t rows);

}  // namespace fp8b
