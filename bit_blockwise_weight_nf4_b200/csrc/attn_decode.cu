// attn_decode.cu -- attention of a few query rows per sequence over a paged
// 4-bit key/value cache on sm_100a (decode, verified drafts): the tier of
// bnb_attn_4bit for at most 16 rows (queries x grouped heads) per key/value
// head.
//   s_j = scale * sum_b a_k[j, b] * sum_{d in block b} q_d t[k_code[j, d]]
//   o_d = sum_j p_j a_v[j, b(d)] t[v_code[j, d]] / sum_j p_j,  p_j = exp(s_j - m)
// over the tokens j a row sees; t is the 16-entry code table.
//
// Design.
//  * The cache is read once: every warp walks tiles of kTile tokens of one
//    (sequence, key/value head), codes straight from global memory into
//    registers one tile ahead, with its own running maximum and sums; the
//    CTA's warps join in shared memory at the end of a segment.
//  * Products run on mma.sync m16n8k16 (fp16 in, fp32 sums) with the cache as
//    the A operand -- 16 tokens of K, or 16 dimensions of V -- and up to 8
//    rows of q or p as B, so that no multiply is spent on padding to 16 rows.
//    The scores leave the first product token-major; movmatrix turns them
//    into the B operand of the second.
//  * The block scales never touch the codes: a_k multiplies the block's
//    partial dot product, a_v the weights p.  So the decode of a code is a
//    lookup in a constant table, done two codes (one byte) at a time in a
//    256-entry table of fp16 pairs in shared memory, replicated for the 32
//    banks so that lookups never conflict: one byte permute forms the
//    address, one 32-bit load gives an operand register.  (The linear kernels
//    look up scaled values by byte permutes, ~2.5 integer operations per
//    code; this is ~0.75 and half a load.)
//  * Precision: q in bf16 is scaled by a power of two per row into fp16
//    without loss (28 binades below the row's largest stay exact); the table
//    is multiplied by the constant that brings its fp16 roundings to 6e-5 of
//    a value's size; weights p a_v are scaled by the running power of two of
//    the block's largest a_v, to at most 2^15, so they stay normal fp16 down
//    to 2^-29 of it.  For fp16 outputs, whose last place is finer than such a
//    weight's rounding, the weights are split into two fp16 terms.
//  * Work is split evenly: the tiles of all (sequence, head) pairs form one
//    line that is cut into equal runs, one per CTA; a run's first and last
//    pair may be shared with its neighbours, whose partial results (fp32, in
//    the workspace) a second kernel joins in the order of the tokens, so
//    results repeat bit for bit.
#include "common.cuh"
#include "kvcache.h"
#include "kernels.h"

namespace bnb4 {
namespace {

struct DecodeArgs {
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
  int row_tiles;  // row tiles per (sequence, head); > 1 only without `split`
  int split;      // the line of tiles is cut into equal runs
  FastDiv page;
  float scale_log2;  // softmax scale * log2(e)
  float* ws;
  int* err;
};

// ------------------------------------------------------------ sequences
// One row tile of one sequence: its rows, and the tokens any of them sees.
struct Span {
  int q0, n, rows, r0;  // first query row of the sequence, its queries, this tile's rows
  int len, first;       // cached tokens; position of query 0
  int lo, base, end, tiles;  // first token seen, the same rounded down to 16, end
};

template <int RT, int TILE>
__device__ __forceinline__ Span span_of(const DecodeArgs& a, int b, int rt) {
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

// ------------------------------------------------------------ primitives
__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                        uint32_t a3, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 "
      "{%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t a) {
  uint32_t d;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
  return d;
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

// The fp16 pair of a code byte: {t[byte >> 4], t[byte & 15]} from the table
// at shared address 64 KB, entry `byte` in 256 bytes, one copy per bank.
// lane_base: bytes {4 * lane, 0, 1, 0}; the permute puts byte I of w between.
template <int I>
__device__ __forceinline__ uint32_t pair_of(uint32_t w, uint32_t lane_base) {
  uint32_t at, v;
  asm("prmt.b32 %0, %1, %2, %3;" : "=r"(at) : "r"(w), "r"(lane_base), "n"(0x7604 | (I << 4)));
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(at));
  return v;
}

__device__ __forceinline__ uint32_t smem_addr(const void* p) {
  return static_cast<uint32_t>(__cvta_generic_to_shared(p));
}

constexpr uint32_t kTableAt = 0x10000;   // shared address of the pair table
constexpr uint32_t kJoinAt = 0x20000;    // and of the warps' partial outputs
// The code table times this constant rounds to fp16 with a root mean square
// error of 6.2e-5 of the values' (1.6e-4 as it stands); FP4's magnitudes
// times 6 are E2M1's, exact.
constexpr float kNf4Scale = 1.67768975f;
constexpr float kFp4Scale = 6.0f;

__device__ __forceinline__ void build_table(int qtype, int warps) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int c = lane & 15;
  const float v = qtype == kQtNF4 ? __fmul_rn(nf4_value(c), kNf4Scale)
                                  : rintf(__fmul_rn(code_value(kQtFP4, c), 12.0f)) * 0.5f;
  const uint32_t h = pack_f16x2(v, 0.0f) & 0xffffu;
  for (int e = warp; e < 256; e += warps) {
    const uint32_t hi = __shfl_sync(0xffffffffu, h, e >> 4);
    const uint32_t lo = __shfl_sync(0xffffffffu, h, e & 15);
    asm volatile("st.shared.u32 [%0], %1;" ::"r"(kTableAt + 256u * e + 4u * lane),
                 "r"(hi | lo << 16)
                 : "memory");
  }
}

template <int BYTES>
struct Chunk {  // 4, 8 or 16 bytes of codes
  uint32_t w[BYTES / 4];
  __device__ __forceinline__ void load(const uint8_t* p) {
    if constexpr (BYTES == 16) {
      const uint4 v = ldg_stream_v4(p);
      w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
    } else if constexpr (BYTES == 8) {
      asm volatile("ld.global.nc.L1::no_allocate.v2.u32 {%0,%1}, [%2];"
                   : "=r"(w[0]), "=r"(w[1])
                   : "l"(p));
    } else {
      asm volatile("ld.global.nc.L1::no_allocate.u32 %0, [%1];" : "=r"(w[0]) : "l"(p));
    }
  }
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int i = 0; i < BYTES / 4; ++i) w[i] = 0u;
  }
};

// NB scales of one cache row (2, 4 or 8 bytes)
template <int NB>
__device__ __forceinline__ void load_scales(const uint16_t* p, uint32_t (&s)[(NB + 1) / 2]) {
  if constexpr (NB == 1) {
    s[0] = __ldg(p);
  } else if constexpr (NB == 2) {
    s[0] = __ldg(reinterpret_cast<const uint32_t*>(p));
  } else {
    const uint2 v = __ldg(reinterpret_cast<const uint2*>(p));
    s[0] = v.x;
    s[1] = v.y;
  }
}
template <int F, int NB>
__device__ __forceinline__ float scale_at(const uint32_t (&s)[(NB + 1) / 2], int b) {
  const uint32_t w = s[b / 2];
  return half_to_f32<F>((b & 1) ? w >> 16 : w & 0xffffu);
}

// One warp tile's codes and scales in flight.
template <int D, int NB, int NS>
struct TileRegs {
  Chunk<D / 8> k[NS][2];
  Chunk<D / 16> v[NS][4];
  uint32_t ka[NS][2][(NB + 1) / 2], va[NS][2][(NB + 1) / 2];
};

// Values d .. d + 3 of row r of (sequence, key/value head): v over its sum of
// weights (relative to 2^top).  A row that saw no token has top = -infinity
// and sum 0 (a NaN score leaves a NaN sum) and gives zeros.
template <int F>
__device__ __forceinline__ void store_row(const DecodeArgs& a, const Span& sp, int h, int r, int d,
                                          const float4& v, float top, float sum) {
  const int i = r / a.group, hh = r - i * a.group;
  const bool sees = top != -INFINITY || sum != 0.0f;
  const float inv = 1.0f / sum;
  const int64_t tok = static_cast<int64_t>(sp.q0) + i;
  const int head = h * a.group + hh;
  uint2 w;
  w.x = sees ? pack2<F>(v.x * inv, v.y * inv) : 0u;
  w.y = sees ? pack2<F>(v.z * inv, v.w * inv) : 0u;
  *reinterpret_cast<uint2*>(a.out + tok * a.o_ts + head * a.o_hs + d) = w;
  if (a.lse && d == 0)
    a.lse[tok * (static_cast<int64_t>(a.heads) * a.group) + head] =
        sees ? (top + lg2(sum)) * 0.693147180559945f : -INFINITY;
}

// ------------------------------------------------------------- the kernel
// D, BS: head dimension and block size.  F: the 16-bit type.  NT: 8-row
// groups of the row tile.  NS: 16-token sub-tiles per tile.  W: warps.
template <int D, int BS, int F, int NT, int NS, int W>
__global__ void __launch_bounds__(W * 32, 1) attn_decode_kernel(const DecodeArgs a) {
  constexpr int RT = 8 * NT, TILE = 16 * NS, NB = D / BS;
  constexpr int KS = D / 16;  // k-steps of q.K; m-tiles of the output
  constexpr int SW = BS / 8;  // values of a block per strip
  constexpr bool kSplitP = F == BNB4_F16;
  extern __shared__ uint8_t smem_raw[];
  __shared__ float sm_m[W][RT], sm_l[W][RT], sm_max[RT], sm_sum[RT];
  __shared__ int sm_item[4];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int g = lane >> 2, t = lane & 3;
  const uint32_t lane_base = kTableAt | (4u * lane);
  // the table's fixed place must lie behind the static arrays and inside the
  // dynamic ones (the launch asks for enough); refused here if it does not
  if (smem_addr(smem_raw) > kTableAt || smem_addr(sm_m) >= kTableAt ||
      smem_addr(sm_item) >= kTableAt) {
    if (threadIdx.x == 0) atomicExch(a.err, 1);
    return;
  }
  pdl_trigger();
  build_table(a.qtype, W);
  pdl_wait();

  // -------- this CTA's run of the line of tiles, or its items in turn
  int64_t left;                  // tiles left of the run (split)
  int b = 0, h = 0, rt = 0, tile0 = 0;
  int64_t item = blockIdx.x;     // without split: (rt, h, b) in turn
  const int64_t items = static_cast<int64_t>(a.batch) * a.heads * a.row_tiles;
  if (a.split) {
    if (warp == 0) {
      int64_t total = 0;
      for (int b0 = 0; b0 < a.batch; b0 += 32) {
        const int i = b0 + lane;
        total += i < a.batch ? static_cast<int64_t>(span_of<RT, TILE>(a, i, 0).tiles) : 0;
      }
      total = warp_sum(total) * a.heads;
      const int64_t per = (total + gridDim.x - 1) / gridDim.x;
      const int64_t u0 = per * blockIdx.x;
      const int64_t mine = u0 >= total ? 0 : total - u0 < per ? total - u0 : per;
      int64_t before = 0;
      int fb = 0, fh = 0, ft = 0;
      if (mine > 0) {
        for (int b0 = 0; b0 < a.batch; b0 += 32) {
          const int i = b0 + lane;
          const int tl = i < a.batch ? span_of<RT, TILE>(a, i, 0).tiles : 0;
          int64_t incl = static_cast<int64_t>(tl) * a.heads;
#pragma unroll
          for (int o = 1; o < 32; o <<= 1) {
            const int64_t y = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += y;
          }
          const unsigned past = __ballot_sync(0xffffffffu, before + incl > u0);
          if (past) {
            const int f = __ffs(past) - 1;
            const int tf = __shfl_sync(0xffffffffu, tl, f);
            const int64_t start =
                before + __shfl_sync(0xffffffffu, incl, f) - static_cast<int64_t>(tf) * a.heads;
            const int64_t x = u0 - start;
            fb = b0 + f;
            fh = static_cast<int>(x / tf);
            ft = static_cast<int>(x - static_cast<int64_t>(fh) * tf);
            break;
          }
          before += __shfl_sync(0xffffffffu, incl, 31);
        }
      }
      if (lane == 0) {
        sm_item[0] = fb;
        sm_item[1] = fh;
        sm_item[2] = ft;
        sm_item[3] = static_cast<int>(mine);
      }
    }
    __syncthreads();
    b = sm_item[0], h = sm_item[1], tile0 = sm_item[2];
    left = sm_item[3];
  } else {
    left = 1;
    __syncthreads();
  }

  for (;;) {
    if (a.split) {
      if (left <= 0 || b >= a.batch) break;
    } else {
      if (item >= items) break;
      rt = static_cast<int>(item % a.row_tiles);
      const int64_t x = item / a.row_tiles;
      h = static_cast<int>(x % a.heads);
      b = static_cast<int>(x / a.heads);
      item += gridDim.x;
    }
    const Span sp = span_of<RT, TILE>(a, b, rt);
    if (sp.rows == 0) {  // uniform over the CTA
      if (a.split) ++b, h = 0, tile0 = 0;  // holds no tiles
      continue;
    }
    const int tile1 = !a.split || sp.tiles - tile0 <= left ? sp.tiles
                                                           : tile0 + static_cast<int>(left);

    // ---------------- q: rows g (and g + 8) as the B operand of every k-step
    uint32_t qf[NT][KS][2];
    float qs[NT][2];  // per column 2 t, 2 t + 1: s = (sum of products) * qs, in log2 units
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const int r = sp.r0 + 8 * n + g;
      const bool real = 8 * n + g < sp.rows;
      const int i = r / a.group, hh = r - i * a.group;
      const uint16_t* src = a.q + (static_cast<int64_t>(sp.q0) + i) * a.q_ts +
                            (static_cast<int64_t>(h) * a.group + hh) * a.q_hs;
      uint32_t raw[KS][2];
      uint32_t top = 0;
#pragma unroll
      for (int s = 0; s < KS; ++s)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          // stored place of the pair, and the dimension it holds
          const int p = t * (D / 4) + 4 * s + 2 * e;
          const int strip = p / (D / 8), x = p % (D / 8);
          const int d = (x / SW) * BS + strip * SW + x % SW;
          raw[s][e] = real ? __ldg(reinterpret_cast<const uint32_t*>(src + d)) : 0u;
          const uint32_t m0 = raw[s][e] & 0x7fffu, m1 = (raw[s][e] >> 16) & 0x7fffu;
          top = max(top, max(m0, m1));
        }
      float mul = a.scale_log2;
      if constexpr (F == BNB4_BF16) {
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
        int e = static_cast<int>(top >> 7) - 127;  // exponent of the row's largest
        e = e < -100 ? -100 : e;
        const float f = pow2(14 - e > 126 ? 126 : 14 - e);
        mul *= pow2(e - 14 < -126 ? -126 : e - 14);
#pragma unroll
        for (int s = 0; s < KS; ++s)
#pragma unroll
          for (int x = 0; x < 2; ++x)
            qf[n][s][x] = pack_f16x2(bf16_lo(raw[s][x]) * f, bf16_hi(raw[s][x]) * f);
      } else {
#pragma unroll
        for (int s = 0; s < KS; ++s) qf[n][s][0] = raw[s][0], qf[n][s][1] = raw[s][1];
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
      }
      // a row with an infinite or NaN entry is NaN, whatever its products are
      if (top >= (F == BNB4_BF16 ? 0x7f80u : 0x7c00u)) mul = __int_as_float(0x7fffffff);
      mul *= a.qtype == kQtNF4 ? 1.0f / kNf4Scale : 1.0f / kFp4Scale;
      // columns 2 t and 2 t + 1 are rows held by lanes 4 (2 t) and 4 (2 t + 1)
      qs[n][0] = __shfl_sync(0xffffffffu, mul, 8 * t);
      qs[n][1] = __shfl_sync(0xffffffffu, mul, 8 * t + 4);
    }
    // last token (inclusive) and first each column sees
    int see_hi[NT][2], see_lo[NT][2];
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const int r = 8 * n + 2 * t + c;
        const int pos = sp.first + (sp.r0 + r) / a.group;
        see_hi[n][c] = r >= sp.rows ? -1 : a.causal && pos < sp.len ? pos : sp.len - 1;
        see_lo[n][c] = a.window > 0 ? pos - a.window + 1 : 0;
      }
    // tokens every row sees: tiles inside need no mask
    const int pos0 = sp.first + sp.r0 / a.group;
    const int all_hi = a.causal && pos0 < sp.len ? pos0 : sp.len - 1;
    const int all_lo = a.window > 0 ? sp.first + (sp.r0 + sp.rows - 1) / a.group - a.window + 1 : 0;

    const int32_t* bt = a.block_table + static_cast<int64_t>(b) * a.bt_stride;

    float m[NT][2], l[NT][2];
    float o[KS][NT][4];
    int ve[NB];  // exponent of the largest a_v so far, per block
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int c = 0; c < 2; ++c) m[n][c] = -INFINITY, l[n][c] = 0.0f;
#pragma unroll
    for (int i = 0; i < KS; ++i)
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int c = 0; c < 4; ++c) o[i][n][c] = 0.0f;
#pragma unroll
    for (int i = 0; i < NB; ++i) ve[i] = -100;

    // lane's rows of a sub-tile: MMA row g is token tok_g, row g + 8 is 8 + tok_g
    const int tok_g = (g & 1) * 4 + (g >> 1);

    // page of each sub-tile of tile i (lane s < NS holds sub-tile s's), -1: none
    auto pages_of = [&](int i) {
      int pg = -1;
      if (lane < NS && i < tile1) {
        const int j = sp.base + i * TILE + 16 * lane;
        if (j < sp.end) {
          const uint32_t x = a.page.div(static_cast<uint32_t>(j));
          const int p = __ldg(bt + x);
          if (p >= 0 && p < a.num_pages) pg = p;
        }
      }
      return pg;
    };
    TileRegs<D, NB, NS> cur;
    uint32_t ok_k = 0, ok_v = 0;
    auto row_at = [&](int i, int s, int pg) {
      const uint32_t j = static_cast<uint32_t>(sp.base + i * TILE + 16 * s);
      const uint32_t in = j - a.page.div(j) * a.page.d;
      return (static_cast<int64_t>(pg) * a.heads + h) * a.page.d + in;
    };
    auto load_k = [&](int i, int pages) {
      ok_k = 0;
#pragma unroll
      for (int s = 0; s < NS; ++s) {
        const int pg = __shfl_sync(0xffffffffu, pages, s);
        if (pg >= 0) {
          ok_k |= 1u << s;
          const int64_t row = row_at(i, s, pg) + tok_g;
          cur.k[s][0].load(a.k_codes + row * (D / 2) + t * (D / 8));
          cur.k[s][1].load(a.k_codes + (row + 8) * (D / 2) + t * (D / 8));
          load_scales<NB>(a.k_absmax + row * NB, cur.ka[s][0]);
          load_scales<NB>(a.k_absmax + (row + 8) * NB, cur.ka[s][1]);
        } else {
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            cur.k[s][x].zero();
#pragma unroll
            for (int y = 0; y < (NB + 1) / 2; ++y) cur.ka[s][x][y] = 0u;
          }
        }
      }
    };
    auto load_v = [&](int i, int pages) {
      ok_v = 0;
#pragma unroll
      for (int s = 0; s < NS; ++s) {
        const int pg = __shfl_sync(0xffffffffu, pages, s);
        if (pg >= 0) {
          ok_v |= 1u << s;
          const int64_t row = row_at(i, s, pg);
#pragma unroll
          for (int c = 0; c < 4; ++c)
            cur.v[s][c].load(a.v_codes + (row + 4 * c + t) * (D / 2) + g * (D / 16));
          load_scales<NB>(a.v_absmax + (row + tok_g) * NB, cur.va[s][0]);
          load_scales<NB>(a.v_absmax + (row + tok_g + 8) * NB, cur.va[s][1]);
        } else {
#pragma unroll
          for (int c = 0; c < 4; ++c) cur.v[s][c].zero();
#pragma unroll
          for (int x = 0; x < 2; ++x)
#pragma unroll
            for (int y = 0; y < (NB + 1) / 2; ++y) cur.va[s][x][y] = 0u;
        }
      }
    };

    int i = tile0 + warp;
    int pages = pages_of(i);
    if (i < tile1) {
      load_k(i, pages);
      load_v(i, pages);
    }
    int pages_next = pages_of(i + W);
    for (; i < tile1; i += W) {
      // ------------------------------------------------ scores
      float s[NS][NT][4];
#pragma unroll
      for (int u = 0; u < NS; ++u) {
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int c = 0; c < 4; ++c) s[u][n][c] = 0.0f;
#pragma unroll
        for (int blk = 0; blk < NB; ++blk) {
          float acc[NT][4];
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int c = 0; c < 4; ++c) acc[n][c] = 0.0f;
#pragma unroll
          for (int st = 0; st < KS; ++st) {
            // k-step st: bytes 2 st and 2 st + 1 of the lane's two strips
            if (((st % (KS / 2)) * 4) / SW != blk) continue;
            const uint32_t w0 = cur.k[u][0].w[st / 2], w1 = cur.k[u][1].w[st / 2];
            uint32_t a0, a1, a2, a3;
            if (st % 2 == 0) {
              a0 = pair_of<0>(w0, lane_base), a1 = pair_of<0>(w1, lane_base);
              a2 = pair_of<1>(w0, lane_base), a3 = pair_of<1>(w1, lane_base);
            } else {
              a0 = pair_of<2>(w0, lane_base), a1 = pair_of<2>(w1, lane_base);
              a2 = pair_of<3>(w0, lane_base), a3 = pair_of<3>(w1, lane_base);
            }
#pragma unroll
            for (int n = 0; n < NT; ++n)
              mma_f16(acc[n], a0, a1, a2, a3, qf[n][st][0], qf[n][st][1]);
          }
          // an infinite scale would make every product infinite or NaN; its
          // row's score is NaN
          float k0 = scale_at<F, NB>(cur.ka[u][0], blk), k1 = scale_at<F, NB>(cur.ka[u][1], blk);
          k0 += k0 - k0;
          k1 += k1 - k1;
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            s[u][n][0] = fmaf(acc[n][0], k0, s[u][n][0]);
            s[u][n][1] = fmaf(acc[n][1], k0, s[u][n][1]);
            s[u][n][2] = fmaf(acc[n][2], k1, s[u][n][2]);
            s[u][n][3] = fmaf(acc[n][3], k1, s[u][n][3]);
          }
        }
      }
      const uint32_t ok = ok_k;
      // the next tile's keys are on their way while this one's weights form
      if (i + W < tile1) load_k(i + W, pages_next);

      const int j0 = sp.base + i * TILE;
      const bool masked =
          ok != (1u << NS) - 1 || j0 < all_lo || j0 + TILE - 1 > all_hi;  // warp-uniform
      float av[NS][2][NB];
#pragma unroll
      for (int u = 0; u < NS; ++u)
#pragma unroll
        for (int x = 0; x < 2; ++x)
#pragma unroll
          for (int blk = 0; blk < NB; ++blk) av[u][x][blk] = scale_at<F, NB>(cur.va[u][x], blk);
      float top[NT][2];
#pragma unroll
      for (int n = 0; n < NT; ++n) top[n][0] = m[n][0], top[n][1] = m[n][1];
#pragma unroll
      for (int u = 0; u < NS; ++u)
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            float v = s[u][n][c] * qs[n][c & 1];
            if (masked) {
              const int j = j0 + 16 * u + tok_g + 8 * (c >> 1);
              if (!((ok >> u) & 1u) || j > see_hi[n][c & 1] || j < see_lo[n][c & 1]) v = -INFINITY;
            }
            s[u][n][c] = v;
            top[n][c & 1] = fmaxf(top[n][c & 1], v);
          }
      if (masked) {  // scales of tokens that no row sees may be anything
#pragma unroll
        for (int u = 0; u < NS; ++u)
#pragma unroll
          for (int x = 0; x < 2; ++x)
          {
            const int j = j0 + 16 * u + tok_g + 8 * x;
            if (!((ok >> u) & 1u) || j >= sp.end || j < sp.lo)
#pragma unroll
              for (int blk = 0; blk < NB; ++blk) av[u][x][blk] = 0.0f;
          }
      }
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int c = 0; c < 2; ++c)
#pragma unroll
          for (int x = 4; x <= 16; x <<= 1)
            top[n][c] = fmaxf(top[n][c], __shfl_xor_sync(0xffffffffu, top[n][c], x));
      // running exponents of the value scales, and the factor that brings a
      // weight times its scale to at most 2^15
      float vn[NB];
      bool grew = false;
      float vgrow[NB];
#pragma unroll
      for (int blk = 0; blk < NB; ++blk) {
        uint32_t x = 0;
#pragma unroll
        for (int u = 0; u < NS; ++u)
#pragma unroll
          for (int y = 0; y < 2; ++y) {
            const uint32_t bits = __float_as_uint(av[u][y][blk]);
            x = max(x, bits < 0x7f800000u ? bits : 0u);  // infinite ones stay infinite
          }
        x = __reduce_max_sync(0xffffffffu, x);
        const int e = static_cast<int>(x >> 23) - 127;
        vgrow[blk] = 1.0f;
        if (e > ve[blk]) {
          const int d = ve[blk] - e;
          vgrow[blk] = d < -126 ? 0.0f : pow2(d);
          ve[blk] = e;
          grew = true;
        }
        vn[blk] = pow2(14 - ve[blk]);
#pragma unroll
        for (int u = 0; u < NS; ++u) av[u][0][blk] *= vn[blk], av[u][1][blk] *= vn[blk];
      }
      bool up = grew;
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int c = 0; c < 2; ++c) up = up || top[n][c] > m[n][c];
      if (__any_sync(0xffffffffu, up)) {
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            const float f = top[n][c] > m[n][c] ? ex2(m[n][c] - top[n][c]) : 1.0f;
            m[n][c] = top[n][c];
            l[n][c] *= f;
#pragma unroll
            for (int x = 0; x < KS; ++x) {
              const float fo = f * vgrow[(2 * x) / SW];
              o[x][n][c] *= fo;
              o[x][n][c + 2] *= fo;
            }
          }
      }
      // ------------------------------------------------ weights and values
#pragma unroll
      for (int u = 0; u < NS; ++u) {
        float p[NT][4];
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            const float mm = m[n][c & 1];
            p[n][c] = ex2(s[u][n][c] - (mm == -INFINITY ? 0.0f : mm));
            l[n][c & 1] += p[n][c];
          }
        uint32_t pb[NB][NT][2], pl[NB][NT][2];
#pragma unroll
        for (int blk = 0; blk < NB; ++blk)
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int x = 0; x < 2; ++x) {
              float y0 = p[n][2 * x] * av[u][x][blk], y1 = p[n][2 * x + 1] * av[u][x][blk];
              if (masked) {  // 0 * infinity of a token that another row sees
                y0 = s[u][n][2 * x] == -INFINITY ? 0.0f : y0;
                y1 = s[u][n][2 * x + 1] == -INFINITY ? 0.0f : y1;
              }
              const uint32_t hi = pack_f16x2(y0, y1);
              pb[blk][n][x] = transpose8x8(hi);
              if constexpr (kSplitP)
                pl[blk][n][x] = transpose8x8(pack_f16x2(
                    y0 - half_to_f32<BNB4_F16>(hi & 0xffffu), y1 - half_to_f32<BNB4_F16>(hi >> 16)));
            }
#pragma unroll
        for (int wd = 0; wd < D / 64; ++wd) {
          // word wd of the lane's strip for its 4 tokens: bytes of the codes
          // of two tokens (even values; odd values)
          const uint32_t w0 = cur.v[u][0].w[wd], w1 = cur.v[u][1].w[wd];
          const uint32_t w2 = cur.v[u][2].w[wd], w3 = cur.v[u][3].w[wd];
          const uint32_t ev0 = (w0 & 0xf0f0f0f0u) | ((w1 >> 4) & 0x0f0f0f0fu);
          const uint32_t od0 = ((w0 << 4) & 0xf0f0f0f0u) | (w1 & 0x0f0f0f0fu);
          const uint32_t ev1 = (w2 & 0xf0f0f0f0u) | ((w3 >> 4) & 0x0f0f0f0fu);
          const uint32_t od1 = ((w2 << 4) & 0xf0f0f0f0u) | (w3 & 0x0f0f0f0fu);
          auto mtile = [&](int x, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3) {
            const int blk = (2 * x) / SW;
#pragma unroll
            for (int n = 0; n < NT; ++n) {
              mma_f16(o[x][n], a0, a1, a2, a3, pb[blk][n][0], pb[blk][n][1]);
              if constexpr (kSplitP)
                mma_f16(o[x][n], a0, a1, a2, a3, pl[blk][n][0], pl[blk][n][1]);
            }
          };
          mtile(4 * wd, pair_of<0>(ev0, lane_base), pair_of<0>(od0, lane_base),
                pair_of<0>(ev1, lane_base), pair_of<0>(od1, lane_base));
          mtile(4 * wd + 1, pair_of<1>(ev0, lane_base), pair_of<1>(od0, lane_base),
                pair_of<1>(ev1, lane_base), pair_of<1>(od1, lane_base));
          mtile(4 * wd + 2, pair_of<2>(ev0, lane_base), pair_of<2>(od0, lane_base),
                pair_of<2>(ev1, lane_base), pair_of<2>(od1, lane_base));
          mtile(4 * wd + 3, pair_of<3>(ev0, lane_base), pair_of<3>(od0, lane_base),
                pair_of<3>(ev1, lane_base), pair_of<3>(od1, lane_base));
        }
      }
      if (i + W < tile1) load_v(i + W, pages_next);
      pages_next = pages_of(i + 2 * W);
    }

    // ---------------------------------------------------- join the warps
    const int busy = tile1 - tile0 < W ? tile1 - tile0 : W;  // warps with a tile
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
#pragma unroll
        for (int x = 4; x <= 16; x <<= 1) l[n][c] += __shfl_xor_sync(0xffffffffu, l[n][c], x);
        if (g == 0) {
          sm_m[warp][8 * n + 2 * t + c] = m[n][c];
          sm_l[warp][8 * n + 2 * t + c] = l[n][c];
        }
      }
    __syncthreads();
    if (threadIdx.x < RT) {
      float top = -INFINITY;
      for (int w = 0; w < busy; ++w) top = fmaxf(top, sm_m[w][threadIdx.x]);
      const float ref = top == -INFINITY ? 0.0f : top;
      float sum = 0.0f;
      for (int w = 0; w < busy; ++w) sum += sm_l[w][threadIdx.x] * ex2(sm_m[w][threadIdx.x] - ref);
      sm_max[threadIdx.x] = top;
      sm_sum[threadIdx.x] = sum;
    }
    __syncthreads();
    const float cinv = a.qtype == kQtNF4 ? 1.0f / kNf4Scale : 1.0f / kFp4Scale;
    const uint32_t mine = kJoinAt + static_cast<uint32_t>(warp) * (RT * D * 4);
    if (warp < busy) {
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          const int r = 8 * n + 2 * t + c;
          const float top = sm_max[r];
          const float f = ex2(m[n][c] - (top == -INFINITY ? 0.0f : top)) * cinv;
#pragma unroll
          for (int x = 0; x < KS; ++x) {
            const int blk = (2 * x) / SW;
            const int d = blk * BS + g * SW + (2 * x) % SW;
            const float back = pow2(ve[blk] - 14);
            asm volatile("st.shared.v2.f32 [%0], {%1, %2};" ::"r"(mine + 4u * (r * D + d)),
                         "f"(o[x][n][c] * f * back), "f"(o[x][n][c + 2] * f * back)
                         : "memory");
          }
        }
    }
    __syncthreads();
    const bool whole = tile0 == 0 && tile1 == sp.tiles;
    // partial results: slot 0 continues the run before, slot 1 goes on in the next
    float* part = a.ws + (static_cast<int64_t>(blockIdx.x) * 2 + (tile0 == 0 ? 1 : 0)) *
                             (RT * D + 2 * RT);
    for (int e = threadIdx.x; e < sp.rows * (D / 4); e += W * 32) {
      const int r = e / (D / 4), d = (e % (D / 4)) * 4;
      float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
      for (int w = 0; w < busy; ++w) {
        float4 y;
        asm volatile("ld.shared.v4.f32 {%0,%1,%2,%3}, [%4];"
                     : "=f"(y.x), "=f"(y.y), "=f"(y.z), "=f"(y.w)
                     : "r"(kJoinAt + 4u * ((w * RT + r) * D + d)));
        v.x += y.x, v.y += y.y, v.z += y.z, v.w += y.w;
      }
      if (whole) {
        store_row<F>(a, sp, h, sp.r0 + r, d, v, sm_max[r], sm_sum[r]);
      } else {
        *reinterpret_cast<float4*>(part + r * D + d) = v;
        if (d == 0) {
          part[RT * D + r] = sm_max[r];
          part[RT * D + RT + r] = sm_sum[r];
        }
      }
    }
    __syncthreads();  // the shared arrays are free for the next segment
    if (a.split) {
      left -= tile1 - tile0;
      tile0 = 0;
      if (++h == a.heads) h = 0, ++b;
    }
  }
}

// Joins the partial results of the pairs that several runs share: CTA i takes
// the pair that begins in run i and goes on in run i + 1.
template <int D, int F, int NT, int NS>
__global__ void __launch_bounds__(256) attn_join_kernel(const DecodeArgs a) {
  constexpr int RT = 8 * NT, TILE = 16 * NS;
  __shared__ int sm_item[5];
  pdl_wait();
  const int lane = threadIdx.x & 31;
  const int64_t run = blockIdx.x;
  if (threadIdx.x < 32) {
    int64_t total = 0;
    for (int b0 = 0; b0 < a.batch; b0 += 32) {
      const int i = b0 + lane;
      total += i < a.batch ? static_cast<int64_t>(span_of<RT, TILE>(a, i, 0).tiles) : 0;
    }
    total = warp_sum(total) * a.heads;
    const int64_t per = (total + gridDim.x - 1) / gridDim.x;
    const int64_t u0 = per * run, u1 = u0 + per < total ? u0 + per : total;
    int found = 0, fb = 0, fh = 0;
    int64_t last_run = 0, before = 0;
    if (u1 > u0) {
      for (int b0 = 0; b0 < a.batch; b0 += 32) {
        const int i = b0 + lane;
        const int tl = i < a.batch ? span_of<RT, TILE>(a, i, 0).tiles : 0;
        int64_t incl = static_cast<int64_t>(tl) * a.heads;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int64_t y = __shfl_up_sync(0xffffffffu, incl, o);
          if (lane >= o) incl += y;
        }
        const unsigned past = __ballot_sync(0xffffffffu, before + incl > u1 - 1);
        if (past) {
          const int f = __ffs(past) - 1;
          const int tf = __shfl_sync(0xffffffffu, tl, f);
          const int64_t start =
              before + __shfl_sync(0xffffffffu, incl, f) - static_cast<int64_t>(tf) * a.heads;
          fb = b0 + f;
          fh = static_cast<int>((u1 - 1 - start) / tf);
          const int64_t s0 = start + static_cast<int64_t>(fh) * tf;  // the pair's first tile
          const int64_t s1 = s0 + tf;
          found = s0 >= u0 && s1 > u1;
          last_run = (s1 - 1) / per;
          break;
        }
        before += __shfl_sync(0xffffffffu, incl, 31);
      }
    }
    if (lane == 0) {
      sm_item[0] = found;
      sm_item[1] = fb;
      sm_item[2] = fh;
      sm_item[3] = static_cast<int>(last_run);
    }
  }
  __syncthreads();
  if (!sm_item[0]) return;
  const int b = sm_item[1], h = sm_item[2], last = sm_item[3];
  const Span sp = span_of<RT, TILE>(a, b, 0);
  constexpr int64_t kPart = RT * D + 2 * RT;
  const int64_t first_part = 2 * run + 1;
  for (int e = threadIdx.x; e < sp.rows * (D / 4); e += blockDim.x) {
    const int r = e / (D / 4), d = (e % (D / 4)) * 4;
    float top = a.ws[first_part * kPart + RT * D + r];
    for (int64_t x = run + 1; x <= last; ++x)
      top = fmaxf(top, a.ws[2 * x * kPart + RT * D + r]);
    const float ref = top == -INFINITY ? 0.0f : top;
    float sum = 0.0f;
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int64_t x = run; x <= last; ++x) {
      const float* part = a.ws + (x == run ? first_part : 2 * x) * kPart;
      const float f = ex2(part[RT * D + r] - ref);
      const float4 y = *reinterpret_cast<const float4*>(part + r * D + d);
      sum = fmaf(part[RT * D + RT + r], f, sum);
      v.x = fmaf(y.x, f, v.x), v.y = fmaf(y.y, f, v.y);
      v.z = fmaf(y.z, f, v.z), v.w = fmaf(y.w, f, v.w);
    }
    store_row<F>(a, sp, h, r, d, v, top, sum);
  }
}

// ------------------------------------------------------------------- host
constexpr int kMaxRuns = 192;  // bound of the grid, hence of the workspace

template <int NT>
constexpr int warps_of() { return NT == 1 ? 16 : 12; }
constexpr int kSub = 2;  // 16-token sub-tiles per warp tile

template <int D, int BS, int F, int NT>
cudaError_t launch_t(const DecodeArgs& a, int grid, cudaStream_t s) {
  constexpr int W = warps_of<NT>(), RT = 8 * NT;
  constexpr int kSmem = static_cast<int>(kJoinAt) + W * RT * D * 4;
  auto kern = attn_decode_kernel<D, BS, F, NT, kSub, W>;
  cudaError_t e =
      cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
  if (e != cudaSuccess) return e;
  e = launch_kernel(kern, dim3(grid), dim3(W * 32), kSmem, s, programmatic_after_kernel(s), a);
  if (e != cudaSuccess || !a.split) return e;
  return launch_kernel(attn_join_kernel<D, F, NT, kSub>, dim3(grid), dim3(256), 0, s, true, a);
}

template <int D, int BS, int F>
cudaError_t launch_f(const DecodeArgs& a, int rows, int grid, cudaStream_t s) {
  return rows <= 8 ? launch_t<D, BS, F, 1>(a, grid, s) : launch_t<D, BS, F, 2>(a, grid, s);
}

}  // namespace

size_t attn_workspace_bytes(const bnb4_attn& a) {
  const int64_t rows = static_cast<int64_t>(a.max_q_len) * (a.n_heads / a.cache->n_kv_heads);
  if (rows > 16) return 0;
  const size_t rt = rows <= 8 ? 8 : 16;
  return sizeof(float) * 2 * kMaxRuns * rt * (static_cast<size_t>(a.cache->head_dim) + 2);
}

cudaError_t launch_attn(const bnb4_attn& p, int num_sms, int* err, cudaStream_t s) {
  const bnb4_kv_cache& c = *p.cache;
  DecodeArgs a = {};
  a.q = static_cast<const uint16_t*>(p.q);
  a.out = static_cast<uint16_t*>(p.out);
  a.lse = p.lse;
  a.q_ts = p.q_stride_t, a.q_hs = p.q_stride_h;
  a.o_ts = p.out_stride_t, a.o_hs = p.out_stride_h;
  a.k_codes = c.k_codes, a.v_codes = c.v_codes;
  a.k_absmax = static_cast<const uint16_t*>(c.k_absmax);
  a.v_absmax = static_cast<const uint16_t*>(c.v_absmax);
  a.block_table = p.block_table, a.bt_stride = p.block_table_stride;
  a.seq_lens = p.seq_lens, a.cu_q = p.cu_seqlens_q;
  a.total_q = p.total_q;
  a.batch = p.batch, a.heads = c.n_kv_heads, a.group = p.n_heads / c.n_kv_heads;
  a.max_q = p.max_q_len;
  a.num_pages = static_cast<int>(c.num_pages);
  a.bt_width = p.block_table_width;
  a.causal = p.causal, a.window = p.window, a.qtype = c.qtype;
  a.page = make_div(static_cast<uint32_t>(c.page_size));
  a.scale_log2 = p.scale * 1.44269504088896f;
  a.ws = static_cast<float*>(p.workspace);
  a.err = err;
  const int64_t rows = static_cast<int64_t>(a.max_q) * a.group;
  const int rt = rows <= 8 ? 8 : 16;
  const int warps = rows <= 8 ? warps_of<1>() : warps_of<2>();
  a.row_tiles = static_cast<int>((rows + rt - 1) / rt);
  // Whole pairs in turn where no pair has more than a tile per warp (a cut
  // would only add the join), else the line of tiles cut into equal runs.
  const int64_t span = a.window > 0 && static_cast<int64_t>(a.window) + a.max_q + 15 < p.max_seq_len
                           ? a.window + a.max_q + 15
                           : p.max_seq_len;
  a.split = a.row_tiles == 1 && span > 16 * kSub * warps;
  const int64_t items = static_cast<int64_t>(a.batch) * a.heads * a.row_tiles;
  const int sms = num_sms < kMaxRuns ? num_sms : kMaxRuns;
  const int grid = a.split || items > sms ? sms : static_cast<int>(items);
#define BNB4_ATTN(DV, BSV)                                                             \
  return c.dtype == BNB4_F16 ? launch_f<DV, BSV, BNB4_F16>(a, rt, grid, s)             \
                             : launch_f<DV, BSV, BNB4_BF16>(a, rt, grid, s);
  if (c.head_dim == 128) {
    if (c.blocksize == 128) { BNB4_ATTN(128, 128) }
    if (c.blocksize == 64) { BNB4_ATTN(128, 64) }
    BNB4_ATTN(128, 32)
  }
  if (c.blocksize == 64) { BNB4_ATTN(64, 64) }
  BNB4_ATTN(64, 32)
#undef BNB4_ATTN
}

}  // namespace bnb4
