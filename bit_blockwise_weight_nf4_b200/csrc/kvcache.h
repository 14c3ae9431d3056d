// kvcache.h -- internal interface of the 4-bit key/value cache kernels
// (kv_cache.cu, attn_decode.cu, attn_prefill.cu).  Not part of the public ABI.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "bnb4.h"

namespace bnb4 {

// Division of n < 2^31 by a constant 1 <= d < 2^31: with s = ceil(log2 d) and
// m = ceil(2^(31 + s) / d), floor(n m / 2^(31 + s)) = floor(n / d), since the
// excess e = m d - 2^(31 + s) < d <= 2^s keeps n e < 2^(31 + s).
struct FastDiv {
  uint32_t d, mul, shift;
#ifdef __CUDACC__
  __device__ __forceinline__ uint32_t div(uint32_t n) const {
    return static_cast<uint32_t>((static_cast<uint64_t>(n) * mul) >> shift);
  }
#endif
};

inline FastDiv make_div(uint32_t d) {
  uint32_t s = 0;
  while ((1ull << s) < d) ++s;
  return FastDiv{d, static_cast<uint32_t>(((1ull << (31 + s)) + d - 1) / d), 31 + s};
}

// Rows of k and v into, or out of, the slots of a cache.  k, v: element (t,
// h, 0) at t * ts + h * hs.
struct KvRows {
  const void *k, *v;
  int64_t k_ts, k_hs, v_ts, v_hs;
};
cudaError_t launch_kv_write(const KvRows& rows, int64_t tokens, const int64_t* slots,
                            const bnb4_kv_cache& c, int num_sms, cudaStream_t s);
cudaError_t launch_kv_read(const bnb4_kv_cache& c, const int64_t* slots, int64_t tokens,
                           const KvRows& rows, int out_dtype, int num_sms, cudaStream_t s);

// Attention over the cache; see bnb_attn_4bit for the arguments.
size_t attn_workspace_bytes(const bnb4_attn& a);
// wait_limit_ns (0: the usual limit) and withhold != 0 are the failure-detection
// diagnostic: CTA 0's first wait runs out.
cudaError_t launch_attn(const bnb4_attn& a, int num_sms, int* err, cudaStream_t s,
                        uint64_t wait_limit_ns = 0, int withhold = 0);

}  // namespace bnb4
