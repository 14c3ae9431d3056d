// kv_cache.cu -- rows of keys and values into the slots of a 4-bit cache and
// back (sm_100a).
//
// A cache row is one head's D values of one token: blocks of BS consecutive
// values, each quantized as bnb_quantize_4bit does (a = max|x|, r = RN(1/a),
// code = midpoints strictly below RN(x r)), the scale a kept in the cache's
// 16-bit type, which holds a maximum of that type's own values exactly.
//
// Layout.  The row's codes lie in 8 strips: strip s holds, block after block,
// values [s w, (s + 1) w) of each block, w = BS / 8 (one block per row: the
// natural order).  The attention kernel hands whole strips to lanes -- two of
// a K row, one of a V row -- and so reads every row with one wide load per
// lane while each lane still holds its share of every block, whose scale
// then multiplies a partial sum instead of each value.
//
// Both kernels are bound by HBM: 2 D bytes of 16-bit values and D / 2 + 2 D /
// BS bytes of cache per row.  A lane owns 8 values (16 bytes) of a row, so D
// / 8 lanes hold a row and the block maximum is an xor-shuffle among BS / 8
// of them; a unit of some rows is in flight per lane, all of one token, whose
// slot is looked up once.  Reading, the next unit's rows are loaded before this
// one's are decoded (its slot a unit earlier still): the latency of two loads
// in a row was most of the time (65536 tokens of 32 heads of 128, bf16: 390 us
// without, 264 us with, 5,140 GB/s, replayed in a graph; 280 to 290 us, 4,700 to
// 4,850 GB/s, on inputs that are new each time).  Writing, whose work per value is longer,
// that gained nothing.  Table lookups are warp shuffles (the table is one entry
// per lane: no shared memory to fill, which a 16-token call would wait for):
// two per value to quantize, one to decode.  Writing 2048 tokens of 32 heads of
// 128 takes 20 us, where the traffic needs 7: the quantizer's instructions.
#include "common.cuh"
#include "kvcache.h"

namespace bnb4 {
namespace {

constexpr int kThreads = 256;
constexpr int kWriteRows = 2, kReadRows = 4;  // rows in flight per lane

// v in [-1, 1] is bucketed as j = rint(14.4 v) + 15 (1 .. 29) with one FMA
// whose integer lands in the mantissa bits; lane j of the warp holds bucket
// j's entry.  Buckets are 0.0695 wide and decision points at least 0.08
// apart, so a bucket widened by 1e-3 on each side holds at most one.  Lane 31
// is where the canonical NaN lands: code 0, as in bnb_quantize_4bit.
constexpr float kPerUnit = 14.4f;
constexpr int kCenter = 15;
constexpr float kMagic = 12582912.0f;  // 1.5 * 2^23

// A bucket's decision point (+inf: none), the code below it, and what the point
// adds to the code (NF4: one; FP4: the upper half of `codes`).  FP4's negative points are
// stored as the float below, so that "v > point" decides v >= -m (a tie goes
// to the smaller magnitude).
struct Bucket {
  float point;
  int32_t codes;
};

__device__ __forceinline__ float midpoint(float a, float b) {
  return __fmul_rn(__fadd_rn(a, b), 0.5f);
}

__device__ Bucket bucket_of_lane(int qt, int lane) {
  Bucket e{__int_as_float(0x7f800000), 0};
  const float c = static_cast<float>(lane - kCenter) / kPerUnit;
  const float lo = c - 0.5f / kPerUnit - 1e-3f, hi = c + 0.5f / kPerUnit + 1e-3f;
  if (lane == 31) return e;
  if (qt == kQtNF4) {
    int below = 0;
#pragma unroll
    for (int i = 0; i < 15; ++i) {
      const float m = midpoint(nf4_value(i), nf4_value(i + 1));
      if (m < lo)
        ++below;
      else if (m <= hi)
        e.point = m;
    }
    e.codes = below;
  } else {
    // the magnitude of the bucket's end nearer zero, and whether a point is inside
    uint32_t m_lo = 0, m_hi = 0;  // magnitudes at the bucket's lower and upper end
    const float a_lo = fabsf(lo), a_hi = fabsf(hi);
#pragma unroll
    for (int i = 0; i < 7; ++i) {
      const float m = midpoint(fp4_magnitude(i), fp4_magnitude(i + 1));
      m_lo += m < a_lo ? 1u : 0u;
      m_hi += m < a_hi ? 1u : 0u;
      if (m >= lo && m <= hi) e.point = m;
      if (-m >= lo && -m <= hi) e.point = __int_as_float(__float_as_int(-m) + 1);
    }
    const int c_lo = static_cast<int>(lo < 0.0f && m_lo != 0 ? m_lo + 8u : m_lo);
    const int c_hi = static_cast<int>(hi < 0.0f && m_hi != 0 ? m_hi + 8u : m_hi);
    e.codes = (c_hi - c_lo) * 65536 | c_lo;
  }
  return e;
}

// codes * 16 + the code of v
template <int QT>
__device__ __forceinline__ uint32_t push_code(uint32_t codes, float v, const Bucket& mine) {
  const int j = __float_as_int(__fmaf_rn(v, kPerUnit, kMagic + kCenter));
  const float point = __shfl_sync(0xffffffffu, mine.point, j);
  const int32_t c = __shfl_sync(0xffffffffu, mine.codes, j);
  if constexpr (QT == kQtNF4) {
    codes = codes * 16u + static_cast<uint32_t>(c);
    if (v > point) ++codes;
  } else {
    codes = codes * 16u + static_cast<uint32_t>(c & 0xffff);
    if (v > point) codes += static_cast<uint32_t>(c >> 16);
  }
  return codes;
}

// Where the 8 codes of values 8 c .. 8 c + 7 lie in a row: 4 bytes at `at`,
// or (BS = 32: the chunk spans two strips) 2 bytes there and 2 a strip on.
template <int D, int BS>
__device__ __forceinline__ int code_byte(int c) {
  constexpr int w = BS / 8;
  if constexpr (D == BS) return 4 * c;
  const int b = 8 * c / BS, o = 8 * c % BS;
  return (o / w) * (D / 16) + b * (w / 2) + (o % w) / 2;
}

template <int D, int BS>
__device__ __forceinline__ void store_codes(uint8_t* row, int c, uint32_t p) {
  uint8_t* at = row + code_byte<D, BS>(c);
  if constexpr (BS == 32 && D > BS) {
    *reinterpret_cast<uint16_t*>(at) = static_cast<uint16_t>(p);
    *reinterpret_cast<uint16_t*>(at + D / 16) = static_cast<uint16_t>(p >> 16);
  } else {
    *reinterpret_cast<uint32_t*>(at) = p;
  }
}
template <int D, int BS>
__device__ __forceinline__ uint32_t load_codes(const uint8_t* row, int c) {
  const uint8_t* at = row + code_byte<D, BS>(c);
  if constexpr (BS == 32 && D > BS)
    return __ldg(reinterpret_cast<const uint16_t*>(at)) |
           static_cast<uint32_t>(__ldg(reinterpret_cast<const uint16_t*>(at + D / 16))) << 16;
  else
    return __ldg(reinterpret_cast<const uint32_t*>(at));
}

struct KvArgs {
  KvRows rows;
  const int64_t* slots;
  uint8_t *k_codes, *v_codes;
  uint16_t *k_absmax, *v_absmax;
  FastDiv per_token, page;  // units of a token; page size
  uint32_t n_units;         // a unit: some rows of a token per lane
  int heads, qtype;
  int64_t n_slots;
};

// A unit's token and its place in the cache: row 0 of its page's head 0 plus its
// row in the page (rows of the next head are a page size on), or -1: the token
// has no slot and is left out.
struct Unit {
  uint32_t t;
  int x0;  // first of the token's 2 * heads rows: keys, then values
  int64_t row;
};
__device__ __forceinline__ int64_t slot_of(const KvArgs& a, uint32_t u) {
  return u < a.n_units ? __ldg(a.slots + a.per_token.div(u)) : -1;
}
__device__ __forceinline__ Unit unit_of(const KvArgs& a, uint32_t u, int64_t slot, int rows) {
  Unit r;
  r.t = a.per_token.div(u);
  r.x0 = static_cast<int>(u - r.t * a.per_token.d) * rows;
  r.row = -1;
  if (slot >= 0 && slot < a.n_slots) {
    const uint32_t pg = a.page.div(static_cast<uint32_t>(slot));
    r.row = static_cast<int64_t>(pg) * a.heads * a.page.d +
            (static_cast<uint32_t>(slot) - pg * a.page.d);
  }
  return r;
}

template <int D, int BS, int F, int QT>
__global__ void __launch_bounds__(kThreads) kv_write_kernel(const KvArgs a) {
  constexpr int kRows = kWriteRows;
  constexpr int LPR = D / 8;      // lanes per row
  constexpr int RPW = 32 / LPR;   // rows per warp and step
  constexpr int LPB = BS / 8;     // lanes per block
  pdl_trigger();
  const int lane = threadIdx.x & 31, c = lane % LPR;
  const Bucket mine = bucket_of_lane(QT, lane);
  pdl_wait();
  const uint32_t warps = gridDim.x * (kThreads / 32);
  const uint32_t warp = blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
  auto load = [&](const Unit& n, uint4 (&x)[kRows]) {
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      const int r = n.x0 + i * RPW + lane / LPR;
      const bool v = r >= a.heads;
      const int h = v ? r - a.heads : r;
      const uint16_t* src = static_cast<const uint16_t*>(v ? a.rows.v : a.rows.k);
      const int64_t ts = v ? a.rows.v_ts : a.rows.k_ts, hs = v ? a.rows.v_hs : a.rows.k_hs;
      x[i] = n.row >= 0 && r < 2 * a.heads ? ldg_stream_v4(src + n.t * ts + h * hs + 8 * c)
                                           : make_uint4(0, 0, 0, 0);
    }
  };
  for (uint32_t u = warp; u < a.n_units; u += warps) {
    const Unit n = unit_of(a, u, slot_of(a, u), RPW * kRows);
    uint4 x[kRows];
    load(n, x);
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      const uint32_t w[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
      float e[8];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if constexpr (F == BNB4_BF16) {
          e[2 * j] = bf16_lo(w[j]);
          e[2 * j + 1] = bf16_hi(w[j]);
        } else {
          e[2 * j] = half_to_f32<F>(w[j] & 0xffffu);
          e[2 * j + 1] = half_to_f32<F>(w[j] >> 16);
        }
      }
      float m = 0.0f;
#pragma unroll
      for (int j = 0; j < 8; ++j) m = fmaxf(m, fabsf(e[j]));  // drops NaN, as the quantizer does
#pragma unroll
      for (int o = LPB / 2; o >= 1; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
      const float inv = m == 0.0f ? 0.0f : __frcp_rn(m);
#pragma unroll
      for (int j = 0; j < 8; ++j) e[j] = __fmul_rn(e[j], inv);
      // only a subnormal scale's reciprocal can leave [-1, 1] (or be
      // infinite); every decision point is inside, and NaN stays NaN
      if (__any_sync(0xffffffffu, m < 0x1p-120f)) {
#pragma unroll
        for (int j = 0; j < 8; ++j) e[j] = e[j] > 1.0f ? 1.0f : e[j] < -1.0f ? -1.0f : e[j];
      }
      uint32_t codes = 0;
#pragma unroll
      for (int j = 3; j >= 0; --j) {  // byte j = code[2 j] << 4 | code[2 j + 1]
        codes = push_code<QT>(codes, e[2 * j], mine);
        codes = push_code<QT>(codes, e[2 * j + 1], mine);
      }
      const int r = n.x0 + i * RPW + lane / LPR;
      if (n.row >= 0 && r < 2 * a.heads) {
        const bool v = r >= a.heads;
        const int64_t row = n.row + static_cast<int64_t>(v ? r - a.heads : r) * a.page.d;
        store_codes<D, BS>((v ? a.v_codes : a.k_codes) + row * (D / 2), c, codes);
        if (c % LPB == 0)
          (v ? a.v_absmax : a.k_absmax)[row * (D / BS) + c / LPB] =
              static_cast<uint16_t>(pack2<F>(m, 0.0f));
      }
    }
  }
}

// OT: BNB4_F32, BNB4_BF16 or BNB4_F16
template <int D, int BS, int F, int OT>
__global__ void __launch_bounds__(kThreads) kv_read_kernel(const KvArgs a) {
  constexpr int kRows = kReadRows, LPR = D / 8;
  constexpr int RPW = 32 / LPR;
  constexpr int LPB = BS / 8;
  pdl_trigger();
  const int lane = threadIdx.x & 31, c = lane % LPR;
  // both halves of the warp hold the table: a lookup's index may carry one
  // bit more than the code
  const float mine = code_value_of(a.qtype, lane & 15);
  pdl_wait();
  const uint32_t warps = gridDim.x * (kThreads / 32);
  const uint32_t warp = blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
  auto load = [&](const Unit& n, uint32_t (&w)[kRows], uint32_t (&s)[kRows]) {
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      const int r = n.x0 + i * RPW + lane / LPR;
      const bool v = r >= a.heads;
      const int64_t row = n.row + static_cast<int64_t>(v ? r - a.heads : r) * a.page.d;
      w[i] = s[i] = 0u;
      if (n.row >= 0 && r < 2 * a.heads) {
        w[i] = load_codes<D, BS>((v ? a.v_codes : a.k_codes) + row * (D / 2), c);
        s[i] = __ldg((v ? a.v_absmax : a.k_absmax) + row * (D / BS) + c / LPB);
      }
    }
  };
  if (warp >= a.n_units) return;
  Unit n = unit_of(a, warp, slot_of(a, warp), RPW * kRows);
  uint32_t w[kRows], s[kRows], wn[kRows], sn[kRows];
  load(n, w, s);
  int64_t slot = slot_of(a, warp + warps);
  for (uint32_t u = warp; u < a.n_units; u += warps) {
    const Unit next = unit_of(a, u + warps, slot, RPW * kRows);
    load(next, wn, sn);
    slot = slot_of(a, u + 2 * warps);
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      const float m = half_to_f32<F>(s[i]);
      float e[8];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        e[2 * j] = __fmul_rn(__shfl_sync(0xffffffffu, mine, w[i] >> (8 * j + 4)), m);
        e[2 * j + 1] = __fmul_rn(__shfl_sync(0xffffffffu, mine, w[i] >> (8 * j)), m);
      }
      const int r = n.x0 + i * RPW + lane / LPR;
      const bool v = r >= a.heads;
      const int h = v ? r - a.heads : r;
      void* base = const_cast<void*>(v ? a.rows.v : a.rows.k);
      w[i] = wn[i];
      s[i] = sn[i];
      if (n.row < 0 || r >= 2 * a.heads || base == nullptr) continue;  // null: not asked for
      const int64_t at = n.t * (v ? a.rows.v_ts : a.rows.k_ts) +
                         h * (v ? a.rows.v_hs : a.rows.k_hs) + 8 * c;
      if constexpr (OT == BNB4_F32) {
        float4* dst = reinterpret_cast<float4*>(static_cast<float*>(base) + at);
        dst[0] = make_float4(e[0], e[1], e[2], e[3]);
        dst[1] = make_float4(e[4], e[5], e[6], e[7]);
      } else {
        *reinterpret_cast<uint4*>(static_cast<uint16_t*>(base) + at) =
            make_uint4(pack2<OT>(e[0], e[1]), pack2<OT>(e[2], e[3]), pack2<OT>(e[4], e[5]),
                       pack2<OT>(e[6], e[7]));
      }
    }
    n = next;
  }
}

KvArgs args_of(const KvRows& rows, int64_t tokens, const int64_t* slots, const bnb4_kv_cache& c,
               int rows_in_flight) {
  KvArgs a;
  a.rows = rows;
  a.slots = slots;
  a.k_codes = c.k_codes;
  a.v_codes = c.v_codes;
  a.k_absmax = static_cast<uint16_t*>(c.k_absmax);
  a.v_absmax = static_cast<uint16_t*>(c.v_absmax);
  const int per_unit = 32 / (c.head_dim / 8) * rows_in_flight;
  const int units = (2 * c.n_kv_heads + per_unit - 1) / per_unit;
  a.per_token = make_div(static_cast<uint32_t>(units));
  a.page = make_div(static_cast<uint32_t>(c.page_size));
  a.n_units = static_cast<uint32_t>(tokens * units);
  a.heads = c.n_kv_heads;
  a.qtype = c.qtype;
  a.n_slots = c.num_pages * c.page_size;
  return a;
}

// As many CTAs as the units fill (a unit per warp), 8 per SM at most (2048
// threads).
unsigned grid_for(const KvArgs& a, int num_sms) {
  const int64_t want = (static_cast<int64_t>(a.n_units) + kThreads / 32 - 1) / (kThreads / 32);
  const int64_t most = static_cast<int64_t>(num_sms) * 8;
  return static_cast<unsigned>(want < most ? want : most);
}

}  // namespace

#define BNB4_KV_SHAPES(CALL)                  \
  if (c.head_dim == 128) {                    \
    if (c.blocksize == 128) { CALL(128, 128) } \
    if (c.blocksize == 64) { CALL(128, 64) }  \
    CALL(128, 32)                             \
  }                                           \
  if (c.blocksize == 64) { CALL(64, 64) }     \
  CALL(64, 32)

cudaError_t launch_kv_write(const KvRows& rows, int64_t tokens, const int64_t* slots,
                            const bnb4_kv_cache& c, int num_sms, cudaStream_t s) {
  const KvArgs a = args_of(rows, tokens, slots, c, kWriteRows);
  const dim3 grid(grid_for(a, num_sms)), block(kThreads);
  const bool prog = programmatic_after_kernel(s), nf4 = c.qtype == kQtNF4;
#define BNB4_WRITE(DV, BSV)                                                                    \
  return c.dtype == BNB4_F16                                                                   \
             ? launch_kernel(nf4 ? kv_write_kernel<DV, BSV, BNB4_F16, kQtNF4>                  \
                                 : kv_write_kernel<DV, BSV, BNB4_F16, kQtFP4>,                 \
                             grid, block, 0, s, prog, a)                                       \
             : launch_kernel(nf4 ? kv_write_kernel<DV, BSV, BNB4_BF16, kQtNF4>                 \
                                 : kv_write_kernel<DV, BSV, BNB4_BF16, kQtFP4>,                \
                             grid, block, 0, s, prog, a);
  BNB4_KV_SHAPES(BNB4_WRITE)
#undef BNB4_WRITE
}

cudaError_t launch_kv_read(const bnb4_kv_cache& c, const int64_t* slots, int64_t tokens,
                           const KvRows& rows, int out_dtype, int num_sms, cudaStream_t s) {
  const KvArgs a = args_of(rows, tokens, slots, c, kReadRows);
  const dim3 grid(grid_for(a, num_sms)), block(kThreads);
  const bool prog = programmatic_after_kernel(s);
#define BNB4_READ_T(DV, BSV, FV)                                                              \
  switch (out_dtype) {                                                                        \
    case BNB4_F32:                                                                            \
      return launch_kernel(kv_read_kernel<DV, BSV, FV, BNB4_F32>, grid, block, 0, s, prog, a); \
    case BNB4_F16:                                                                            \
      return launch_kernel(kv_read_kernel<DV, BSV, FV, BNB4_F16>, grid, block, 0, s, prog, a); \
    default:                                                                                  \
      return launch_kernel(kv_read_kernel<DV, BSV, FV, BNB4_BF16>, grid, block, 0, s, prog, a); \
  }
#define BNB4_READ(DV, BSV)                               \
  if (c.dtype == BNB4_F16) {                             \
    BNB4_READ_T(DV, BSV, BNB4_F16)                       \
  } else {                                               \
    BNB4_READ_T(DV, BSV, BNB4_BF16)                      \
  }
  BNB4_KV_SHAPES(BNB4_READ)
#undef BNB4_READ
#undef BNB4_READ_T
}

}  // namespace bnb4
