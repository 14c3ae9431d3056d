// attn.cuh -- what the attention kernels over the 4-bit cache share: their
// arguments, the span of tokens that a tile of rows sees, the code table's
// scaling, and where a row's result goes.
#pragma once

#include "common.cuh"
#include "kvcache.h"

namespace bnb4 {

struct AttnArgs {
  const uint16_t* q;
  uint16_t* out;
  float* lse;
  int64_t q_ts, q_hs, o_ts, o_hs;
  const uint8_t *k_codes, *v_codes;
  const uint16_t *k_absmax, *v_absmax;
  const int32_t* block_table;
  int64_t bt_stride;
  const int32_t *seq_lens, *cu_q;
  int64_t total_q;
  int batch, heads, group, max_q, num_pages, bt_width, causal, window, qtype;
  int row_tiles;  // the kernel for many rows: row tiles per (sequence, head)
  int split;      // the other one: the line of tiles is cut into equal runs
  FastDiv page;
  float scale_log2;  // softmax scale * log2(e)
  float* ws;
  int* err;
  uint64_t wait_limit_ns;
  int withhold;  // failure-detection diagnostic: CTA 0 waits for what never comes
};

// The tensor-core kernel for tiles of 2 x 128 rows (attn_prefill.cu): `rows`
// query rows per (sequence, key/value head) at most, `span` tokens seen at
// most by a row (by which the work is split).
size_t attn_prefill_workspace(const AttnArgs& a, int head_dim, int64_t rows, int64_t span,
                              int num_sms);
cudaError_t launch_attn_prefill(AttnArgs& a, const bnb4_kv_cache& c, int64_t rows, int64_t span,
                                int num_sms, cudaStream_t s);

namespace {

// ------------------------------------------------------------ sequences
// One row tile of one sequence: its rows, and the tokens any of them sees.
struct Span {
  int q0, n, rows, r0;  // first query row of the sequence, its queries, this tile's rows
  int len, first;       // cached tokens; position of query 0
  int lo, base, end, tiles;  // first token seen, the same rounded down to 16, end
};

template <int RT, int TILE>
__device__ __forceinline__ Span span_of(const AttnArgs& a, int b, int rt) {
  Span s;
  if (a.cu_q) {
    const int64_t lo = a.cu_q[b], hi = a.cu_q[b + 1];
    const int64_t c = lo < 0 ? 0 : lo > a.total_q ? a.total_q : lo;
    const int64_t e = hi < c ? c : hi > a.total_q ? a.total_q : hi;
    s.q0 = static_cast<int>(c);
    s.n = static_cast<int>(e - c);
  } else {
    s.q0 = b * a.max_q;
    s.n = a.max_q;
  }
  const int64_t room = static_cast<int64_t>(a.bt_width) * a.page.d;
  int len = a.seq_lens[b];
  len = len < 0 ? 0 : len;
  s.len = len > room ? static_cast<int>(room) : len;
  s.first = s.len - s.n;
  const int n = s.n < a.max_q ? s.n : a.max_q;  // rows past max_q are not computed
  s.r0 = rt * RT;
  int rows = n * a.group - s.r0;
  s.rows = rows < 0 ? 0 : rows > RT ? RT : rows;
  s.lo = s.base = s.end = s.tiles = 0;
  if (s.rows > 0) {
    const int i0 = s.r0 / a.group, i1 = (s.r0 + s.rows - 1) / a.group;
    const int last = s.first + i1;  // position of the last row
    s.end = a.causal && last + 1 < s.len ? last + 1 : s.len;
    if (s.end < 0) s.end = 0;
    int lo = a.window > 0 ? s.first + i0 - a.window + 1 : 0;
    if (lo < 0) lo = 0;
    s.lo = lo;
    s.base = lo & ~15;
    // at least one tile, so that rows that see nothing are still written
    s.tiles = s.end > s.base ? (s.end - s.base + TILE - 1) / TILE : 1;
  }
  return s;
}

__device__ __forceinline__ int64_t warp_sum(int64_t x) {
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float lg2(float x) {
  float y;
  asm("lg2.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// 2^e for -126 <= e <= 127
__device__ __forceinline__ float pow2(int e) { return __int_as_float((e + 127) << 23); }

// A score (in binades) below which half a step of its last place, 2^-8, leaves a
// weight's size as it is.
constexpr float kFarScore = 65536.0f;

// The code table times this constant rounds to fp16 within 3.1e-4 of a value,
// exactly at the block's largest (1 and -1), with a root mean square error of
// 3.6e-5 of the scale (as it stands: 8.1e-5); of the constants with exact ends
// it leaves the least error in attention over normal keys (simulated: 2.0e-4
// of the output against 4.3e-4).  FP4's magnitudes times 6 are E2M1's, exact.
constexpr float kNf4Scale = 1613.0f / 1024.0f;
constexpr float kFp4Scale = 6.0f;
__device__ __forceinline__ float scaled_code(int qtype, int c) {
  const float v = code_value_of(qtype, c);
  // E2M1's magnitudes are multiples of a half
  return qtype == kQtNF4 ? __fmul_rn(v, kNf4Scale) : rintf(__fmul_rn(v, 2.0f * kFp4Scale)) * 0.5f;
}

// Where row r of (sequence, key/value head) goes, divided by its sum of weights
// (relative to 2^top).  A row that saw no token has top = -infinity and sum 0
// (a NaN score leaves a NaN sum) and gives zeros.
template <int F>
struct RowOut {
  uint16_t* at;
  float inv;
  bool sees;
  __device__ __forceinline__ RowOut(const AttnArgs& a, const Span& sp, int h, int r, float top,
                                    float sum, bool write_lse) {
    const int i = r / a.group, hh = r - i * a.group;
    const int64_t tok = static_cast<int64_t>(sp.q0) + i;
    const int head = h * a.group + hh;
    sees = top != -INFINITY || sum != 0.0f;
    inv = 1.0f / sum;
    at = a.out + tok * a.o_ts + head * a.o_hs;
    if (write_lse && a.lse)
      a.lse[tok * (static_cast<int64_t>(a.heads) * a.group) + head] =
          sees ? (top + lg2(sum)) * 0.693147180559945f : -INFINITY;
  }
  __device__ __forceinline__ void pair(int d, float x, float y) const {
    *reinterpret_cast<uint32_t*>(at + d) = sees ? pack2<F>(x * inv, y * inv) : 0u;
  }
};

}  // namespace
}  // namespace bnb4
