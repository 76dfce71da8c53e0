// kv_common.cuh -- what the kernels of the paged FP8 KV cache share: a sequence's place in the
// call and the checks of what only the device sees.
#pragma once

#include "common.cuh"
#include "kernels.h"

namespace fp8b {

// Sequence b of a call: its rows [first, first + n) of the call's tensors and its length
// in the cache.  ok is false when cu_q or the length cannot be right (nothing of the
// sequence may then be touched).
struct Sequence {
    int32_t first, n, kv_len;
    bool ok;
};

__device__ __forceinline__ Sequence sequence_of(const KvArgs& c, int32_t b, int64_t max_kv) {
    Sequence s;
    const int32_t lo = c.cu_q ? __ldg(c.cu_q + b) : b;
    const int32_t hi = c.cu_q ? __ldg(c.cu_q + b + 1) : b + 1;
    s.kv_len = __ldg(c.kv_lens + b);
    s.ok = lo >= 0 && hi >= lo && hi <= c.tokens && hi - lo <= c.max_q && s.kv_len >= 0 && s.kv_len <= max_kv &&
           s.kv_len <= c.max_pages * c.page_size;
    s.first = lo;
    s.n = hi - lo;
    return s;
}

}  // namespace fp8b
