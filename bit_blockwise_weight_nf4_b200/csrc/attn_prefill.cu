// attn_prefill.cu -- attention of many query rows over a paged 4-bit
// key/value cache on sm_100a (chunks of prompts): the tier of bnb_attn_4bit
// for more than 16 rows (queries x grouped heads) per key/value head.
//
//   s_ij = scale * sum_d q_id t[k_code] a_k,  p_ij = exp(s_ij - m_i)
//   o_id = sum_j p_ij t[v_code] a_v / sum_j p_ij
// over the tokens j that row i sees, the running maximum m_i and the sums kept
// in fp32 while the tokens pass once.
//
// Two matrix products on the tensor cores (tcgen05, fp16 in, fp32 sums in
// tensor memory) around an online softmax, for tiles of 2 x 128 rows against
// 128 tokens.
//
// What bounds it (2 prompts of 2048 tokens, 32 heads of 128, bf16, NF4 blocks of
// 64: 127 us, 543 TFLOP/s of the visible pairs' products; the products alone
// would take 41 us).  A tile of 256 x 128 takes 5,100 cycles.  The softmax warps
// are busy all of them but 580 -- 2,550 in the exponentials, which the two
// warps of a scheduler share, the rest in the latencies of the loads from
// tensor memory, maxima and hand-overs --, the warps that issue the products
// wait 2,000 of them, and the decode's 4 + 4 warps 700 to 1,700.  The products
// themselves need 2,700: with 64 columns at a time an operand of 6 KB is read
// per 50 cycles, all that shared memory gives.  An item's start and end (page
// table, first rows, q, first tile, output) cost 9 us, of which 3.5 items per
// SM each pay their share.
// Measured and not taken: more splits of the tokens than fill the SMs once
// (slower by the join), the next half's scores loaded during this half's
// weights (154 us: 96 registers a thread do not hold both), wholly unrolled
// decoding and L2 prefetches of the codes (no difference), a CTA that walks
// several items (slower: its turns bind the roles to one another).
//
// Roles of a CTA's 18 warps (one CTA per SM):
//  * warps 0-3 and 4-7: the softmax of row tile 0 and 1, one row per thread.
//    Tokens are taken 64 at a time, in two halves of the scores' columns: a
//    half's next scores are computed while the other half's weights form, so
//    the softmax does not wait for the products.  The running
//    maximum is only raised when it grows by more than 8 binades; until then
//    weights exceed one, and the sums in tensor memory need no rescaling.
//    The weights go back to tensor memory, over the scores, as the A operand
//    of the second product.
//  * warps 8-11: the keys.  Thread r owns token r of the tile: 64 codes a
//    64-byte row in registers one tile ahead, looked up two at a time (a byte)
//    in a table of fp16 pairs in shared memory, times the block's scale, into
//    the swizzled K-major operand.
//  * warps 12-15: the values.  Thread u owns 8 tokens x 8 or 16 values; bytes
//    of two tokens' codes of the same value are put together first, so that
//    the operand (values as rows, tokens as K) is again written 8 codes and 16
//    bytes at a time.
//  * warps 16 and 17 issue the products of row tile 0 and 1: the sums of a half
//    and the scores of the next one to take its columns.  (A wait, a commit
//    and a product each cost the issuing warp around a hundred cycles: done by
//    a softmax warp, or by one warp for both row tiles, they set the pace.)
// Two row tiles share a CTA because the decode of a tile of keys and values
// takes as long as the rest for 128 rows: 148 CTAs with 4352 tokens each take
// 100 us for one row tile and 106 for both.
// The stored order of a row's values is kept for K and q alike (a dot product
// does not care) and undone when the output is written.
//
// Precision.  q as in the decode kernel; keys are rounded to fp16 after
// scaling by the power of two of their tile's largest scale, values by a running
// one, both to at most 2^16, and weights by 2^7 (so at most 2^15): keys and values
// stay normal 24 binades below the largest, whether a row sees that one or not,
// weights 21.  Of bf16 caches an NF4 key is off by the table's rounding and the
// product's, 2.3e-4 of itself in the mean square, which the scores carry into the
// exponent: next to the error of fp32 weights 1.03 times it at scores of a
// standard deviation of 1, 1.14 at 10, 1.41 at 30 (FP4's products are exact:
// 1.01).  For fp16 caches, whose outputs' last place is finer than those
// roundings, keys, values and weights are kept in two fp16 terms (twice the
// products for the scores, three times for the sums; in one term the weights'
// rounding made up to 1.56 times the error of exact fp32 weights).  The prompts
// above take 222 us in fp16.
// Every mbarrier wait is bounded; no TMA load is used.
#include "attn.cuh"
#include "common.cuh"
#include "kernels.h"
#include "kvcache.h"
#include "lut.cuh"
#include "sm100.cuh"

namespace bnb4 {
namespace {

constexpr int TK = 128;        // tokens per decoded tile
constexpr int TH = TK / 2;     // tokens per step of the softmax
constexpr int TR = 128;        // rows per row tile (threads of a softmax group)
constexpr int kRowsCta = 2 * TR;
constexpr int kKeyWarp = 8, kValueWarp = 12, kIssueWarp = 16;
constexpr int kThreads = 18 * 32;
constexpr int kMaxStages = 2;
constexpr int kRing = 4;       // tiles' scalars: see Meta
constexpr float kLazy = 8.0f;  // growth of the maximum that is let pass, in binades
constexpr int kBoost = 7;      // weights are held times 2^kBoost
// Keys and values are held times 2^(top - exponent of the largest scale): NF4's
// table ends at 1.58, FP4's at 6, so at most 5.2e4 in fp16, and normal down to
// 2^-25 of the largest scale.  (A score of 128 such products with q, below 2^16,
// stays below 2^40.)
__host__ __device__ constexpr int held_top(int qtype) { return qtype == kQtNF4 ? 14 : 12; }
constexpr int kHalf = TK * 128;  // 128 rows of 128 bytes

// HL: keys and values are held in two fp16 terms each (fp16 caches: see the
// precision note above), a tile of both at a time instead of two.
template <int D, bool HL>
struct Smem {
  static constexpr int kStages = HL ? 1 : 2;         // decoded tiles of keys, and of values
  static constexpr int kQ = (D / 64) * kHalf;        // one row tile of q
  static constexpr int kKTerm = (D / 64) * kHalf;    // one tile of keys, a term
  static constexpr int kVTerm = (TK / 64) * D * 128; // one tile of values, a term
  static constexpr int kK = kKTerm * (HL ? 2 : 1), kV = kVTerm * (HL ? 2 : 1);
  static constexpr int kOffK = 2 * kQ;
  static constexpr int kOffV = kOffK + kStages * kK;
  static constexpr int kOffTable = kOffV + kStages * kV;
  static constexpr int kOffCtl = kOffTable + 256 * 128;
};

// A tile's scalars, in a ring of 4: tile j + 4's are written after the scores
// of tile j + 1 were complete for both row tiles (k_empty), hence after their
// softmax of tile j -- its readers are done, and a wait never falls two phases
// behind.
struct Meta {
  int key_exp, value_exp;   // keys are held times 2^-key_exp, values 2^(top - value_exp)
  uint8_t present[4];       // per key warp: bit s: its sub-tile s (16 tokens) is cached
  uint32_t bad[4];          // tokens whose value scale is not finite
};

struct Ctl {
  // of a row tile: q is there; a half's scores and its weights are complete;
  // the sums are, but for the last half, and in the end
  uint64_t q_full[2], s_full[2][2], p_full[2][2], o_full[2], done[2];
  uint64_t k_full[kMaxStages], k_empty[kMaxStages], v_full[kMaxStages], v_empty[kMaxStages];
  uint64_t m_full[kRing];
  uint64_t wait_limit_ns;
  uint32_t tmem_base;
  int abort;
  uint32_t top[2][4];  // the key and value warps' largest scales
  Meta meta[kRing];
};

// The products are issued by a whole warp, of which one lane (`one` != 0) acts:
// so descriptors and addresses stay in uniform registers.  A descriptor is
// given by its low word (the address / 16); the high word is a constant.
__device__ __forceinline__ uint64_t desc_at(uint32_t lo) {
  return static_cast<uint64_t>(static_cast<uint32_t>(sw128_desc(0) >> 32)) << 32 | lo;
}
__device__ __forceinline__ uint32_t desc_lo(uint32_t addr) {
  return static_cast<uint32_t>(sw128_desc(addr));
}
__device__ __forceinline__ void umma_ss(uint32_t one, uint32_t d, uint32_t a, uint32_t b,
                                        uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.b32 q, %0, 0;\n\t"
      "setp.ne.b32 p, %5, 0;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%1], %2, %3, %4, p;\n\t}" ::"r"(one),
      "r"(d), "l"(desc_at(a)), "l"(desc_at(b)), "r"(idesc), "r"(accumulate));
}
// the A operand in tensor memory
__device__ __forceinline__ void umma_ts(uint32_t one, uint32_t d, uint32_t a, uint32_t b,
                                        uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.b32 q, %0, 0;\n\t"
      "setp.ne.b32 p, %5, 0;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%1], [%2], %3, %4, p;\n\t}" ::"r"(one),
      "r"(d), "r"(a), "l"(desc_at(b)), "r"(idesc), "r"(accumulate));
}
__device__ __forceinline__ void umma_commit(uint32_t one, uint32_t bar) {
  asm volatile(
      "{\n\t.reg .pred q;\n\t"
      "setp.ne.b32 q, %0, 0;\n\t"
      "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%1];\n\t}" ::"r"(
          one),
      "r"(bar)
      : "memory");
}
__device__ __forceinline__ void tmem_load32(uint32_t at, float (&v)[32]) {
  uint32_t* r = reinterpret_cast<uint32_t*>(v);
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]),
        "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]),
        "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(at));
}
// Loads have arrived: the registers may be used (and are tied to this point).
__device__ __forceinline__ void tmem_load_done(float (&v)[32]) {
  uint32_t* r = reinterpret_cast<uint32_t*>(v);
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]),
                 "+r"(r[6]), "+r"(r[7]), "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]),
                 "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]), "+r"(r[16]), "+r"(r[17]),
                 "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]), "+r"(r[22]), "+r"(r[23]),
                 "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]), "+r"(r[29]),
                 "+r"(r[30]), "+r"(r[31])::"memory");
}
__device__ __forceinline__ void tmem_load16(uint32_t at, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15])
      : "r"(at)
      : "memory");
}
__device__ __forceinline__ void tmem_store16(uint32_t at, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
      "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(at),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
      "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]),
      "r"(r[15])
      : "memory");
}
__device__ __forceinline__ void tmem_store_done() {
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ float max3(float a, float b, float c) {  // drops NaN, as fmaxf
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
// two fp32 values at a time
__device__ __forceinline__ uint64_t pair_f32(float lo, float hi) {
  return static_cast<uint64_t>(__float_as_uint(hi)) << 32 | __float_as_uint(lo);
}
__device__ __forceinline__ float lo_f32(uint64_t x) {
  return __uint_as_float(static_cast<uint32_t>(x));
}
__device__ __forceinline__ float hi_f32(uint64_t x) {
  return __uint_as_float(static_cast<uint32_t>(x >> 32));
}
__device__ __forceinline__ uint64_t fma_f32x2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
__device__ __forceinline__ uint64_t add_f32x2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ uint32_t fma_f16x2(uint32_t a, uint32_t b, uint32_t c) {
  uint32_t d;
  asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
  return d;
}
__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
// The 4 warps of the keys (or the values) meet.
__device__ __forceinline__ void group_sync(int id) {
  asm volatile("bar.sync %0, 128;" ::"r"(id) : "memory");
}
// What mul_f16x2(t, f) rounded away (exact in one fma, but for subnormal
// results), and the table's own residue r times f.
__device__ __forceinline__ uint32_t rest_f16x2(uint32_t t, uint32_t r, uint32_t f, uint32_t y) {
  return fma_f16x2(r, f, fma_f16x2(t, f, y ^ 0x80008000u));
}

// The residues of the table's fp16 roundings, for byte permutes (lut.cuh).
__device__ __forceinline__ Lut make_residues(int qtype) {
  uint32_t P[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const float n0 = __fmul_rn(nf4_value(2 * j), kNf4Scale);
    const float n1 = __fmul_rn(nf4_value(2 * j + 1), kNf4Scale);
    const uint32_t h = pack_f16x2(n0, n1);
    P[j] = qtype == kQtNF4 ? pack_f16x2(__fsub_rn(n0, half_to_f32<BNB4_F16>(h & 0xffffu)),
                                        __fsub_rn(n1, half_to_f32<BNB4_F16>(h >> 16)))
                           : 0u;  // E2M1's magnitudes are exact
  }
  Lut l;
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    l.L[q] = prmt(P[2 * q], P[2 * q + 1], 0x6420);
    l.H[q] = prmt(P[2 * q], P[2 * q + 1], 0x7531);
  }
  return l;
}

// The table of code pairs: entry `byte` holds the fp16 pair {t[byte >> 4],
// t[byte & 15]} (times the table's constant), one copy per bank.
__device__ __forceinline__ void build_pairs(uint32_t at, int qtype, int warp, int warps) {
  const int lane = threadIdx.x & 31, c = lane & 15;
  const float v = scaled_code(qtype, c);
  const uint32_t h = pack_f16x2(v, 0.0f) & 0xffffu;
#pragma unroll 4
  for (int e = warp; e < 256; e += warps) {
    const uint32_t x = __shfl_sync(0xffffffffu, h, e >> 4) | __shfl_sync(0xffffffffu, h, e & 15) << 16;
    asm volatile("st.shared.u32 [%0], %1;" ::"r"(at + 128u * e + 4u * lane), "r"(x) : "memory");
  }
}
// The pair of byte I of w; lane_table: the table's shared address + 4 * lane.
template <int I>
__device__ __forceinline__ uint32_t pair_of(uint32_t w, uint32_t lane_table) {
  uint32_t at, v;
  asm("{\n\t.reg .b32 b;\n\t"
      "prmt.b32 b, %1, 0, %3;\n\t"
      "mad.lo.u32 %0, b, 128, %2;\n\t}"
      : "=r"(at)
      : "r"(w), "r"(lane_table), "n"(0x4440 | I));
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(at));
  return v;
}

// Columns outside lo .. hi, and of sub-tiles (a bit per 16) that are not
// present, are not seen.
__device__ __forceinline__ uint32_t mask_bits(uint32_t present, int lo, int hi) {
  uint32_t k = ((present & 1u) ? 0x0000ffffu : 0u) | ((present & 2u) ? 0xffff0000u : 0u);
  if (lo > 0) k = lo > 31 ? 0u : k & (0xffffffffu << lo);
  if (hi < 31) k = hi < 0 ? 0u : k & (0xffffffffu >> (31 - hi));
  return k;
}
__device__ __forceinline__ void mask32(float (&v)[32], uint32_t present, int lo, int hi) {
  const uint32_t k = mask_bits(present, lo, hi);
#pragma unroll
  for (int x = 0; x < 32; ++x) v[x] = (k >> x) & 1u ? v[x] : -INFINITY;
}

// Stored place x (a multiple of 4) of a row -> the value's number in the row.
template <int D, int BS>
__device__ __forceinline__ constexpr int value_at(int x) {
  constexpr int w = BS / 8;
  const int strip = x / (D / 8), y = x % (D / 8);
  return (y / w) * BS + strip * w + y % w;
}

struct PrefillArgs {
  AttnArgs a;
  int splits;
};

template <int D, int BS, int F>
__global__ void __launch_bounds__(kThreads, 1) attn_prefill_kernel(const PrefillArgs pa) {
  constexpr bool HL = F == BNB4_F16;
  using S = Smem<D, HL>;
  constexpr int NB = D / BS, kStages = S::kStages;
  const AttnArgs& a = pa.a;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  uint8_t* smem = smem_raw + (((raw + 1023u) & ~1023u) - raw);
  Ctl* ctl = reinterpret_cast<Ctl*>(smem + S::kOffCtl);
  __shared__ __align__(16) uint16_t value_scale[NB][TK];  // fp16, of the tile being decoded
  // the same in every lane, in a form the compiler can see
  const int warp = __shfl_sync(0xffffffffu, static_cast<int>(threadIdx.x) >> 5, 0);
  const int lane = threadIdx.x & 31;
  pdl_trigger();
  pdl_wait();

  // this CTA's rows (the tiles with the most tokens first) and tokens
  const int pairs = a.batch * a.heads;
  const int item = static_cast<int>(blockIdx.x) / pa.splits;
  const int split = static_cast<int>(blockIdx.x) - item * pa.splits;
  const int pair = item % pairs;
  const int rt = a.row_tiles - 1 - item / pairs;
  const int h = pair % a.heads, b = pair / a.heads;
  const Span sp = span_of<kRowsCta, TK>(a, b, rt);
  if (sp.rows == 0) return;  // uniform over the CTA
  const int per = (sp.tiles + pa.splits - 1) / pa.splits;
  const int tile0 = split * per < sp.tiles ? split * per : sp.tiles;
  const int tile1 = tile0 + per < sp.tiles ? tile0 + per : sp.tiles;
  // 0: nothing to add (a partial result of no weight)
  const int T = __shfl_sync(0xffffffffu, tile1 - tile0, 0);
  const int nr = __shfl_sync(0xffffffffu, sp.rows > TR ? 2 : 1, 0);
  const int32_t* bt = a.block_table + static_cast<int64_t>(b) * a.bt_stride;
  auto bar = [&](uint64_t& x) { return smem_u32(&x); };

  if (threadIdx.x == 0) {
    for (int r = 0; r < 2; ++r) {
      mbar_init(bar(ctl->s_full[r][0]), 1);
      mbar_init(bar(ctl->s_full[r][1]), 1);
      mbar_init(bar(ctl->o_full[r]), 1);
      mbar_init(bar(ctl->done[r]), 1);
      mbar_init(bar(ctl->q_full[r]), 4);
      mbar_init(bar(ctl->p_full[r][0]), 4);
      mbar_init(bar(ctl->p_full[r][1]), 4);
    }
    for (int s = 0; s < kStages; ++s) {
      mbar_init(bar(ctl->k_full[s]), 4);
      mbar_init(bar(ctl->k_empty[s]), nr);
      mbar_init(bar(ctl->v_full[s]), 4);
      mbar_init(bar(ctl->v_empty[s]), nr);
    }
    for (int s = 0; s < kRing; ++s) mbar_init(bar(ctl->m_full[s]), 8);
    ctl->abort = 0;
    ctl->wait_limit_ns = a.wait_limit_ns;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 0) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     smem_u32(&ctl->tmem_base)),
                 "r"(512));
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
  // Every warp calls this once, when its first loads are on their way: tensor
  // memory, the barriers and the table are there from then on.
  uint32_t tmem = 0;
  auto ready = [&]() {
    asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
    __syncthreads();
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
    tmem = __shfl_sync(0xffffffffu, ctl->tmem_base, 0);
  };
  // columns: scores (and weights over them) of row tile r at 128 r, sums at 256 + 128 r
  auto s_col = [&](int r) { return tmem + 128u * r; };
  auto o_col = [&](int r) { return tmem + 256u + 128u * r; };
  // A warp's bounded wait; once one has given up, all return at once.  Every lane
  // asks for itself: by one lane, with the others waiting for it, prompts of
  // 2048 tokens took 151 us instead of 128.
  auto warp_wait = [&](uint64_t& x, uint32_t parity) {
    wait_short(bar(x), parity, ctl, a.err);
    __syncwarp();
  };

  if (warp < kKeyWarp) {
    // ------------------------------------------------------------ softmax
    const int r = warp >> 2;
    if (r >= nr) {
      ready();
    } else {
      const int row = static_cast<int>(threadIdx.x);  // of the CTA's 256
      const int rr = sp.r0 + row;
      const bool real = row < sp.rows;
      const int i = real ? rr / a.group : 0, hh = real ? rr - i * a.group : 0;
      const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
      float qs = a.scale_log2;
      {  // q, in the stored order, as fp16: D / 8 lanes read a row
        constexpr int kPer = 256 / D, kSteps = 32 / kPer;  // rows per step, steps per warp
        const int64_t mine = (static_cast<int64_t>(sp.q0) + i) * a.q_ts +
                             (static_cast<int64_t>(h) * a.group + hh) * a.q_hs;
        const unsigned reals = __ballot_sync(0xffffffffu, real);
        const int c = lane % (D / 8), sub = lane / (D / 8);  // stored places 8 c .. of a row
        uint32_t top = 0;  // of this thread's own row
        uint8_t* dst = smem + r * S::kQ + ((warp & 3) * 32) * 128 + (c / 8) * kHalf;
        uint4 x[kSteps];
#pragma unroll
        for (int y = 0; y < kSteps; ++y) {
          const int rw = y * kPer + sub;  // of the warp's 32
          const uint16_t* src = a.q + __shfl_sync(0xffffffffu, mine, rw);
          x[y] = make_uint4(0, 0, 0, 0);
          if ((reals >> rw) & 1u) {
            if constexpr (BS >= 64) {
              x[y] = __ldg(reinterpret_cast<const uint4*>(src + value_at<D, BS>(8 * c)));
            } else {
              const uint2 y0 = __ldg(reinterpret_cast<const uint2*>(src + value_at<D, BS>(8 * c)));
              const uint2 y1 =
                  __ldg(reinterpret_cast<const uint2*>(src + value_at<D, BS>(8 * c + 4)));
              x[y] = make_uint4(y0.x, y0.y, y1.x, y1.y);
            }
          }
        }
        ready();
#pragma unroll
        for (int y = 0; y < kSteps; ++y) {
          // the row's largest magnitude, as the pattern of its bits
          uint32_t t = __vmaxu2(__vmaxu2(x[y].x & 0x7fff7fffu, x[y].y & 0x7fff7fffu),
                                __vmaxu2(x[y].z & 0x7fff7fffu, x[y].w & 0x7fff7fffu));
#pragma unroll
          for (int o = D / 16; o >= 1; o >>= 1)
            t = __vmaxu2(t, __shfl_xor_sync(0xffffffffu, t, o));
          t = max(t & 0xffffu, t >> 16);
          uint4 v = x[y];
          if constexpr (F == BNB4_BF16) {
            int e = static_cast<int>(t >> 7) - 127;
            const float f = pow2(14 - (e < -100 ? -100 : e));
            v = make_uint4(pack_f16x2(bf16_lo(v.x) * f, bf16_hi(v.x) * f),
                           pack_f16x2(bf16_lo(v.y) * f, bf16_hi(v.y) * f),
                           pack_f16x2(bf16_lo(v.z) * f, bf16_hi(v.z) * f),
                           pack_f16x2(bf16_lo(v.w) * f, bf16_hi(v.w) * f));
          }
          // a row with an infinite or NaN entry is NaN as a whole: see attn_decode.cu
          if (t >= (F == BNB4_BF16 ? 0x7f80u : 0x7c00u))
            v = make_uint4(0x7fff7fffu, 0x7fff7fffu, 0x7fff7fffu, 0x7fff7fffu);
          const int rw = y * kPer + sub;
          *reinterpret_cast<uint4*>(dst + rw * 128 + (((c & 7) ^ (rw & 7)) << 4)) = v;
          const uint32_t own = __shfl_sync(0xffffffffu, t, (lane % kPer) * (D / 8));
          if (lane / kPer == y) top = own;
        }
        if constexpr (F == BNB4_BF16) {
          int e = static_cast<int>(top >> 7) - 127;
          qs *= pow2((e < -100 ? -100 : e) - 14);
        }
        qs *= a.qtype == kQtNF4 ? 1.0f / kNf4Scale : 1.0f / kFp4Scale;
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        __syncwarp();
        if (lane == 0 && !(a.withhold && blockIdx.x == 0 && warp == 0))
          mbar_arrive(bar(ctl->q_full[r]));
      }
      // what this row sees, and what all rows of the row tile see
      const int pos = sp.first + rr / a.group;
      const int see_hi = !real ? -1 : a.causal && pos < sp.len ? pos : sp.len - 1;
      const int see_lo = a.window > 0 ? pos - a.window + 1 : 0;
      const int last_row = sp.rows < TR * (r + 1) ? sp.rows - 1 : TR * (r + 1) - 1;
      const int pos0 = sp.first + (sp.r0 + TR * r) / a.group;
      const int all_hi = a.causal && pos0 < sp.len ? pos0 : sp.len - 1;
      const int all_lo = a.window > 0 ? sp.first + (sp.r0 + last_row) / a.group - a.window + 1 : 0;

      float m = -INFINITY, l = 0.0f;
      int ve = 0;
      // of the tile: a bit per 16 tokens, tokens whose value scale is not finite, ...
      uint32_t present = 0;
      uint2 bad = make_uint2(0, 0);
      int tve = 0;
      float q2 = 0.0f;
      for (int i2 = 0; i2 < 2 * T; ++i2) {
        const int j = i2 >> 1, hf = i2 & 1;
        const uint32_t at = s_col(r) + lanes + TH * hf;
        const Meta& mt = ctl->meta[j % kRing];
        if (hf == 0) {
          warp_wait(ctl->m_full[j % kRing], (j / kRing) & 1);
          const uint32_t pr = *reinterpret_cast<const uint32_t*>(mt.present);
          present = (pr & 3u) | ((pr >> 6) & 12u) | ((pr >> 12) & 48u) | ((pr >> 18) & 192u);
          bad = make_uint2(mt.bad[0] | mt.bad[1], mt.bad[2] | mt.bad[3]);
          tve = mt.value_exp;
          q2 = qs * pow2(mt.key_exp);
          if (q2 == 0.0f) q2 = 0x1p-126f;  // so that -infinity stays masked
        } else {
          present >>= 4;
          bad.x = bad.y;
        }
        warp_wait(ctl->s_full[r][hf], j & 1);
        asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
        float v[32], w[32];
        tmem_load32(at, v);
        tmem_load32(at + 32, w);
        const int j0 = sp.base + (tile0 + j) * TK + TH * hf;
        const bool masked = (present & 15u) != 15u || j0 < all_lo || j0 + TH - 1 > all_hi;  // warp-uniform
        // columns lo .. hi of the half are inside what the row sees
        const int lo = see_lo - j0, hi = see_hi - j0;
        tmem_load_done(v);
        tmem_load_done(w);
        if (masked) {
          asm volatile("" ::: "memory");  // a branch, not selects on every tile
          mask32(v, present, lo, hi);
          mask32(w, present >> 2, lo - 32, hi - 32);
        }
        float t[4];
#pragma unroll
        for (int x = 0; x < 4; ++x) t[x] = fmaxf(v[x], v[x + 4]);
#pragma unroll
        for (int x = 8; x < 32; x += 8)
#pragma unroll
          for (int y = 0; y < 4; ++y) t[y] = max3(t[y], v[x + y], v[x + y + 4]);
#pragma unroll
        for (int x = 0; x < 32; x += 8)
#pragma unroll
          for (int y = 0; y < 4; ++y) t[y] = max3(t[y], w[x + y], w[x + y + 4]);
        // q2 > 0; a row of NaN scores has no maximum
        const float top = __fmul_rn(fmaxf(max3(t[0], t[1], t[2]), t[3]), q2);
        const bool grow = top > m + kLazy || (m == -INFINITY && top > m);
        const bool shift = i2 > 0 && tve != ve;
        if (__any_sync(0xffffffffu, grow) || shift) {
          const float old = m;
          if (grow) m = top;
          float f = grow ? ex2(old - m) : 1.0f;
          l *= f;
          if (shift) f *= ve - tve < -126 ? 0.0f : pow2(ve - tve);
          if (i2 > 0) {
            // the sums so far, once they are complete: the scores asked for
            // after them are (if any were), or they themselves
            if (i2 + 1 < 2 * T)
              warp_wait(ctl->s_full[r][hf ^ 1], ((i2 + 1) >> 1) & 1);
            else
              warp_wait(ctl->o_full[r], 0);
            asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
#pragma unroll 1
            for (int c = 0; c < D / 16; ++c) {
              uint32_t y[16];
              tmem_load16(o_col(r) + lanes + 16 * c, y);
#pragma unroll
              for (int x = 0; x < 16; ++x) y[x] = __float_as_uint(__uint_as_float(y[x]) * f);
              tmem_store16(o_col(r) + lanes + 16 * c, y);
            }
          }
        }
        ve = tve;
        float ref = m == -INFINITY ? 0.0f : m, mul = q2;
        // Scores so large that half a step of theirs counts: the product is rounded
        // as the maximum's was, before the maximum is taken off, so that weights
        // stay within 2^kLazy (the fma below would leave that half step).
        if (__any_sync(0xffffffffu, fabsf(ref) > kFarScore)) {
          asm volatile("" ::: "memory");  // a branch
#pragma unroll
          for (int x = 0; x < 32; ++x) {
            v[x] = __fsub_rn(__fmul_rn(v[x], q2), ref);
            w[x] = __fsub_rn(__fmul_rn(w[x], q2), ref);
          }
          ref = 0.0f, mul = 1.0f;
        }
        ref -= static_cast<float>(kBoost);
        uint64_t sum2 = 0;  // two sums of the weights
        const uint64_t q22 = pair_f32(mul, mul), ref2 = pair_f32(-ref, -ref);
        uint32_t p[16];
        auto weights = [&](float (&y)[32]) {
#pragma unroll
          for (int x = 0; x < 32; x += 2) {
            const uint64_t z = fma_f32x2(pair_f32(y[x], y[x + 1]), q22, ref2);
            const float e0 = ex2(lo_f32(z)), e1 = ex2(hi_f32(z));
            sum2 = add_f32x2(sum2, pair_f32(e0, e1));
            p[x / 2] = pack_f16x2(e0, e1);
            if constexpr (HL) y[x] = e0, y[x + 1] = e1;
          }
        };
        // what the weights' fp16 rounding left, over the other half of the scores
        auto rest = [&](const float (&y)[32]) {
#pragma unroll
          for (int x = 0; x < 32; x += 2)
            p[x / 2] = pack_f16x2(y[x] - half_to_f32<BNB4_F16>(p[x / 2] & 0xffffu),
                                  y[x + 1] - half_to_f32<BNB4_F16>(p[x / 2] >> 16));
        };
        weights(v);
        tmem_store16(at, p);
        if constexpr (HL) {
          rest(v);
          tmem_store16(at + TH / 2, p);
        }
        weights(w);
        tmem_store16(at + 16, p);
        if constexpr (HL) {
          rest(w);
          tmem_store16(at + TH / 2 + 16, p);
        }
        l += lo_f32(sum2) + hi_f32(sum2);
        // a value that is not finite, of a token that this row sees
        if (bad.x != 0)
          for (int x = 0; x < TH; ++x)
            if ((mt.bad[2 * hf + (x >> 5)] >> (x & 31)) & 1u)
              if (x >= lo && x <= hi) l = __int_as_float(0x7fffffff);
        tmem_store_done();
        asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(ctl->p_full[r][hf]));
      }
      // ---------------------------------------------------------- output
      if (T > 0) {
        warp_wait(ctl->done[r], 0);
        asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
      }
      {
        const float back = pow2(ve - held_top(a.qtype)) *
                           (a.qtype == kQtNF4 ? 1.0f / kNf4Scale : 1.0f / kFp4Scale);
        const float lse_top = m - static_cast<float>(kBoost);
        const bool sees = m != -INFINITY || l != 0.0f;
        float v[32];
        if (pa.splits == 1) {
          const float inv = back / l;
          const int64_t tok = static_cast<int64_t>(sp.q0) + i;
          const int head = h * a.group + hh;
          const int64_t mine = tok * a.o_ts + head * a.o_hs;
          const unsigned reals = __ballot_sync(0xffffffffu, real);
          if (real && a.lse)
            a.lse[tok * (static_cast<int64_t>(a.heads) * a.group) + head] =
                sees ? (lse_top + lg2(l)) * 0.693147180559945f : -INFINITY;
          // rows go through the place that q had (its products are complete), to
          // be written whole by D / 8 lanes each
          uint8_t* stage = smem + r * S::kQ + ((warp & 3) * 32) * 128;
#pragma unroll
          for (int c = 0; c < D / 32; ++c) {
            tmem_load32(o_col(r) + lanes + 32 * c, v);
            tmem_load_done(v);
#pragma unroll
            for (int x = 0; x < 32; x += 8) {
              uint4 w;
              w.x = sees ? pack2<F>(v[x] * inv, v[x + 1] * inv) : 0u;
              w.y = sees ? pack2<F>(v[x + 2] * inv, v[x + 3] * inv) : 0u;
              w.z = sees ? pack2<F>(v[x + 4] * inv, v[x + 5] * inv) : 0u;
              w.w = sees ? pack2<F>(v[x + 6] * inv, v[x + 7] * inv) : 0u;
              const int p = 4 * c + x / 8;  // stored places 8 p ..
              *reinterpret_cast<uint4*>(stage + (p / 8) * kHalf + lane * 128 +
                                        (((p & 7) ^ (lane & 7)) << 4)) = w;
            }
          }
          __syncwarp();
          const int c = lane % (D / 8), sub = lane / (D / 8);
          constexpr int kPer = 256 / D;
#pragma unroll 4
          for (int y = 0; y < 32 / kPer; ++y) {
            const int rw = y * kPer + sub;  // of the warp's 32
            const int64_t at = __shfl_sync(0xffffffffu, mine, rw);
            const uint4 w = *reinterpret_cast<const uint4*>(stage + (c / 8) * kHalf + rw * 128 +
                                                            (((c & 7) ^ (rw & 7)) << 4));
            if ((reals >> rw) & 1u) {
              uint16_t* dst = a.out + at;
              if constexpr (BS >= 64) {
                *reinterpret_cast<uint4*>(dst + value_at<D, BS>(8 * c)) = w;
              } else {
                *reinterpret_cast<uint2*>(dst + value_at<D, BS>(8 * c)) = make_uint2(w.x, w.y);
                *reinterpret_cast<uint2*>(dst + value_at<D, BS>(8 * c + 4)) = make_uint2(w.z, w.w);
              }
            }
          }
        } else {
          // partial sums (in the stored order), then {maximum, sum} per row
          float* part = a.ws + static_cast<int64_t>(blockIdx.x) * kRowsCta * (D + 2);
          if (real) {
            part[kRowsCta * D + 2 * row] = lse_top;
            part[kRowsCta * D + 2 * row + 1] = l;
          }
#pragma unroll
          for (int c = 0; c < D / 32; ++c) {
            if (T > 0) {  // CTA-uniform
              tmem_load32(o_col(r) + lanes + 32 * c, v);
              tmem_load_done(v);
              if (real) {
#pragma unroll
                for (int x = 0; x < 32; x += 4)
                  *reinterpret_cast<float4*>(part + row * D + 32 * c + x) =
                      make_float4(v[x] * back, v[x + 1] * back, v[x + 2] * back, v[x + 3] * back);
              }
            }
          }
        }
      }
    }
  } else if (warp < kIssueWarp) {
    // ------------------------------------------- keys and values: decode
    const bool values = warp >= kValueWarp;
    const int u = static_cast<int>(threadIdx.x) - (values ? kValueWarp : kKeyWarp) * 32;
    const uint32_t lane_table = smem_u32(smem + S::kOffTable) + 4u * lane;
    Lut residues;
    if constexpr (HL) residues = make_residues(a.qtype);
    // a token's page entry, read two tiles ahead (-1: not cached), and its cache
    // row, computed when the entry has arrived
    auto entry_of = [&](int tile, int tok) {
      const int j = sp.base + (tile0 + tile) * TK + tok;
      // whole sub-tiles of 16 tokens are brought in (a page holds them whole)
      return tile < T && (j & ~15) < sp.end ? __ldg(bt + a.page.div(static_cast<uint32_t>(j))) : -1;
    };
    auto row_of = [&](int entry, int tile, int tok) {
      const uint32_t j = static_cast<uint32_t>(sp.base + (tile0 + tile) * TK + tok);
      const uint32_t in = j - a.page.div(j) * a.page.d;
      return entry >= 0 && entry < a.num_pages
                 ? (static_cast<int64_t>(entry) * a.heads + h) * a.page.d + in
                 : static_cast<int64_t>(-1);
    };
    // scales of token u: raw patterns
    const uint16_t* absmax = values ? a.v_absmax : a.k_absmax;
    auto load_scales = [&](int64_t row, uint32_t (&s)[NB]) {
#pragma unroll
      for (int x = 0; x < NB; ++x) s[x] = row >= 0 ? __ldg(absmax + row * NB + x) : 0u;
    };
    // codes: a key thread's whole token (D / 8 words); a value thread's words
    // word0 .. of the 8 tokens of `group`.  8 neighbouring lanes take 8 groups,
    // whose 16-byte pieces of an operand row fall into different banks.
    constexpr int kWords = D / 8, kUnits = D / 64;
    const int group = (lane & 7) + 8 * (warp & 1);
    const int word0 = kUnits * ((lane >> 3) + 4 * ((warp >> 1) & 1));
    uint32_t w[16], wn[16];
    const int first = values ? 8 * group : u;  // the thread's codes start at this token
    auto load_codes = [&](uint32_t (&x)[16], int64_t at) {
      if (!values) {
#pragma unroll
        for (int y = 0; y < kWords / 4; ++y) {
          const uint4 c = at >= 0 ? ldg_stream_v4(a.k_codes + at * (D / 2) + 16 * y)
                                  : make_uint4(0, 0, 0, 0);
          x[4 * y] = c.x, x[4 * y + 1] = c.y, x[4 * y + 2] = c.z, x[4 * y + 3] = c.w;
        }
      } else {
#pragma unroll
        for (int y = 0; y < 8; ++y) {
          const uint8_t* src = a.v_codes + (at + y) * (D / 2) + 4 * word0;
          if constexpr (kUnits == 2) {
            const uint2 c =
                at >= 0 ? __ldg(reinterpret_cast<const uint2*>(src)) : make_uint2(0, 0);
            x[y] = c.x, x[8 + y] = c.y;
          } else {
            x[y] = at >= 0 ? __ldg(reinterpret_cast<const uint32_t*>(src)) : 0u;
          }
        }
      }
    };
    uint32_t sc[NB], scn[NB];
    int64_t row = row_of(entry_of(0, u), 0, u);  // cache row of token u of this tile
    load_scales(row, sc);
    load_codes(w, row_of(entry_of(0, first), 0, first));
    int e1 = entry_of(1, u), c1 = entry_of(1, first);  // the next tile's entries
    build_pairs(smem_u32(smem + S::kOffTable), a.qtype, warp - kKeyWarp, 8);
    ready();
    int run_exp = -100;  // values: exponent of the largest scale so far
    const int top_exp = held_top(a.qtype);
    for (int j = 0; j < T; ++j) {
      const int s = j % kStages;
      // the next tile's loads are on their way while this one is decoded
      const int64_t row1 = row_of(e1, j + 1, u);
      load_scales(row1, scn);
      load_codes(wn, row_of(c1, j + 1, first));
      e1 = entry_of(j + 2, u);
      c1 = entry_of(j + 2, first);

      const int tok = sp.base + (tile0 + j) * TK + u;
      const bool here = row >= 0;
      // scales of tokens that no row sees count as zero
      const bool seen = here && tok >= sp.lo && tok < sp.end;
      float f[NB];
      uint32_t top = 0;
      bool bad = false;
#pragma unroll
      for (int x = 0; x < NB; ++x) {
        const uint32_t bits = seen ? sc[x] : 0u;
        f[x] = half_to_f32<F>(bits);
        const bool finite = bits < (F == BNB4_BF16 ? 0x7f80u : 0x7c00u);
        bad = bad || !finite;
        top = max(top, finite ? bits : 0u);
      }
      top = __reduce_max_sync(0xffffffffu, top);
      if (lane == 0) ctl->top[values][warp & 3] = top;
      group_sync(values ? 2 : 1);
#pragma unroll
      for (int x = 0; x < 4; ++x) top = max(top, ctl->top[values][x]);
      int e = F == BNB4_BF16 ? static_cast<int>(top >> 7) - 127 : static_cast<int>(top >> 10) - 15;
      e = e < -100 ? -100 : e;
      if (values) e = run_exp = e > run_exp ? e : run_exp;
      const float norm = pow2(top_exp - e);
      // fp16 factors; a key row with a scale that is not finite becomes NaN, a
      // value row zero (the rows that see it are made NaN by the softmax)
      uint32_t fac[NB];
#pragma unroll
      for (int x = 0; x < NB; ++x) {
        const float y = bad ? (values ? 0.0f : __int_as_float(0x7fffffff)) : f[x] * norm;
        fac[x] = pack_f16x2(y, y);
      }
      Meta& mt = ctl->meta[j % kRing];
      const unsigned have = __ballot_sync(0xffffffffu, here);
      const unsigned bads = __ballot_sync(0xffffffffu, bad);
      if (values) {
#pragma unroll
        for (int x = 0; x < NB; ++x) value_scale[x][u] = static_cast<uint16_t>(fac[x]);
      }
      if (lane == 0) {
        if (values) {
          mt.bad[warp & 3] = bads;
          if ((warp & 3) == 0) mt.value_exp = e;
        } else {
          mt.present[warp & 3] = static_cast<uint8_t>((have & 1u) | ((have >> 15) & 2u));
          if ((warp & 3) == 0) mt.key_exp = e - top_exp;
        }
        mbar_arrive(bar(ctl->m_full[j % kRing]));
      }
      // the products that read this stage last have completed; all of the
      // group's scales are there
      warp_wait(values ? ctl->v_empty[s] : ctl->k_empty[s], ((j / kStages) & 1) ^ 1);
      group_sync(values ? 2 : 1);
      if (!values) {
        uint8_t* dst = smem + S::kOffK + s * S::kK + u * 128;
#pragma unroll 1
        for (int x0 = 0; x0 < kWords; x0 += 4) {
#pragma unroll
          for (int y = 0; y < 4; ++y) {
            const uint4 v = make_uint4(pair_of<0>(w[y], lane_table), pair_of<1>(w[y], lane_table),
                                       pair_of<2>(w[y], lane_table), pair_of<3>(w[y], lane_table));
            // word x0 + y holds stored places 8 (x0 + y) ..: of one block, or two of
            // 4 values; 4 words are whole strips, so the blocks follow from y
            const int b0 = ((8 * y) % (D / 8)) / (BS / 8), b1 = ((8 * y + 4) % (D / 8)) / (BS / 8);
            const uint4 k = make_uint4(mul_f16x2(v.x, fac[b0]), mul_f16x2(v.y, fac[b0]),
                                       mul_f16x2(v.z, fac[b1]), mul_f16x2(v.w, fac[b1]));
            uint8_t* at = dst + (x0 / 8) * kHalf + ((((x0 & 7) + y) ^ (u & 7)) << 4);
            *reinterpret_cast<uint4*>(at) = k;
            if constexpr (HL) {
              const uint4 r = dq8(residues, w[y]);
              *reinterpret_cast<uint4*>(at + S::kKTerm) = make_uint4(
                  rest_f16x2(v.x, r.x, fac[b0], k.x), rest_f16x2(v.y, r.y, fac[b0], k.y),
                  rest_f16x2(v.z, r.z, fac[b1], k.z), rest_f16x2(v.w, r.w, fac[b1], k.w));
            }
          }
#pragma unroll
          for (int y = 0; y < 12; ++y) w[y] = w[y + 4];
        }
      } else {
        // the 8 tokens are piece group % 8 of half group / 8 of the operand's rows
        uint8_t* half = smem + S::kOffV + s * S::kV + (group / 8) * (D * 128);
#pragma unroll 1
        for (int word = word0; word < word0 + kUnits; ++word) {
          // bytes of two tokens' codes: of the word's even values, and its odd ones
          uint32_t ev[4], od[4];
#pragma unroll
          for (int y = 0; y < 4; ++y) {
            const uint32_t t0 = w[2 * y], t1 = w[2 * y + 1];
            ev[y] = (t0 & 0xf0f0f0f0u) | ((t1 >> 4) & 0x0f0f0f0fu);
            od[y] = ((t0 << 4) & 0xf0f0f0f0u) | (t1 & 0x0f0f0f0fu);
          }
#pragma unroll
          for (int y = 0; y < 8; ++y) w[y] = w[y + 8];
          const int b0 = ((8 * word) % (D / 8)) / (BS / 8);
          uint4 g = *reinterpret_cast<const uint4*>(&value_scale[b0][8 * group]);
          uint8_t* dst = half + 8 * word * 128;
          // row 8 word + y of the operand: the pairs of tokens t[0] .. t[3]
          auto put_row = [&](int y, const uint32_t (&t)[4]) {
            const uint4 v = make_uint4(
                mul_f16x2(pair_of<0>(t[0], lane_table), g.x),
                mul_f16x2(pair_of<0>(t[1], lane_table), g.y),
                mul_f16x2(pair_of<0>(t[2], lane_table), g.z),
                mul_f16x2(pair_of<0>(t[3], lane_table), g.w));
            uint8_t* at = dst + y * 128 + (((group & 7) ^ y) << 4);
            *reinterpret_cast<uint4*>(at) = v;
            if constexpr (HL) {
              // the codes of one byte each, as two of a word's eight
              const uint4 r0 = dq8(residues, (t[0] & 0xffu) | (t[1] & 0xffu) << 8 |
                                                 (t[2] & 0xffu) << 16 | t[3] << 24);
              *reinterpret_cast<uint4*>(at + S::kVTerm) = make_uint4(
                  rest_f16x2(pair_of<0>(t[0], lane_table), r0.x, g.x, v.x),
                  rest_f16x2(pair_of<0>(t[1], lane_table), r0.y, g.y, v.y),
                  rest_f16x2(pair_of<0>(t[2], lane_table), r0.z, g.z, v.z),
                  rest_f16x2(pair_of<0>(t[3], lane_table), r0.w, g.w, v.w));
            }
          };
#pragma unroll 1
          for (int y = 0; y < 8; y += 2) {  // values 8 word + y and the next: byte y / 2
            if (BS == 32 && y == 4)
              g = *reinterpret_cast<const uint4*>(&value_scale[b0 + 1][8 * group]);
            put_row(y, ev);
            put_row(y + 1, od);
#pragma unroll
            for (int x = 0; x < 4; ++x) ev[x] >>= 8, od[x] >>= 8;
          }
        }
      }
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(values ? ctl->v_full[s] : ctl->k_full[s]));
      row = row1;
#pragma unroll
      for (int x = 0; x < NB; ++x) sc[x] = scn[x];
#pragma unroll
      for (int x = 0; x < 16; ++x) w[x] = wn[x];
    }
  } else {
    // ------------------------------------------------------- products
    constexpr uint32_t kBase = (1u << 4) | (static_cast<uint32_t>(TR >> 4) << 24);
    constexpr uint32_t kIdescS = kBase | (static_cast<uint32_t>(TH >> 3) << 17);
    constexpr uint32_t kIdescO = kBase | (static_cast<uint32_t>(D >> 3) << 17);
    const uint32_t q_at = smem_u32(smem), k_at = q_at + S::kOffK, v_at = q_at + S::kOffV;
    // A wait that gives up ends every later one at once, and all loops run on
    // to their end on whatever is there.
    const int r = warp - kIssueWarp;
    const uint32_t one = lane == 0 ? 1u : 0u;
    ready();
    const uint32_t q_lo = desc_lo(q_at + r * S::kQ), k_lo = desc_lo(k_at), v_lo = desc_lo(v_at);
    auto product_s = [&](int i) {  // scores = q * keys: half i & 1 of tile i / 2
      const int j = i >> 1, hf = i & 1;
      if (hf == 0) warp_wait(ctl->k_full[j % kStages], (j / kStages) & 1);
      asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
      const uint32_t k = k_lo + (j % kStages) * (S::kK / 16) + hf * (TH * 128 / 16);
#pragma unroll
      for (int x = 0; x < D / 16; ++x)
        umma_ss(one, s_col(r) + TH * hf, q_lo + (x / 4) * (kHalf / 16) + 2 * (x & 3),
                k + (x / 4) * (kHalf / 16) + 2 * (x & 3), kIdescS, x > 0);
      if constexpr (HL) {
#pragma unroll
        for (int x = 0; x < D / 16; ++x)
          umma_ss(one, s_col(r) + TH * hf, q_lo + (x / 4) * (kHalf / 16) + 2 * (x & 3),
                  k + S::kKTerm / 16 + (x / 4) * (kHalf / 16) + 2 * (x & 3), kIdescS, 1u);
      }
      umma_commit(one, bar(ctl->s_full[r][hf]));
      if (hf) umma_commit(one, bar(ctl->k_empty[j % kStages]));
    };
    auto product_o = [&](int i) {  // sums += weights * values
      const int j = i >> 1, hf = i & 1;
      if (hf == 0) warp_wait(ctl->v_full[j % kStages], (j / kStages) & 1);
      warp_wait(ctl->p_full[r][hf], j & 1);
      asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
      const uint32_t v = v_lo + (j % kStages) * (S::kV / 16) + hf * (D * 128 / 16);
#pragma unroll
      for (int k = 0; k < TH / 16; ++k)
        umma_ts(one, o_col(r), s_col(r) + TH * hf + 8 * k, v + 2 * k, kIdescO, i > 0 || k > 0);
      if constexpr (HL) {
#pragma unroll
        for (int k = 0; k < TH / 16; ++k)
          umma_ts(one, o_col(r), s_col(r) + TH * hf + 8 * k, v + S::kVTerm / 16 + 2 * k, kIdescO,
                  1u);
#pragma unroll
        for (int k = 0; k < TH / 16; ++k)  // the weights' second term
          umma_ts(one, o_col(r), s_col(r) + TH * hf + TH / 2 + 8 * k, v + 2 * k, kIdescO, 1u);
      }
      if (hf) umma_commit(one, bar(ctl->v_empty[j % kStages]));
    };
    if (r < nr && T > 0) {
      warp_wait(ctl->q_full[r], 0);
      product_s(0);
      product_s(1);
      for (int i = 0; i < 2 * T; ++i) {
        product_o(i);
        if (i + 2 < 2 * T)
          product_s(i + 2);
        else
          umma_commit(one, bar(i + 1 < 2 * T ? ctl->o_full[r] : ctl->done[r]));
      }
      // the products in flight finish before tensor memory is given back, also
      // where the softmax warps gave up waiting for them
      if (lane == 0) wait_drain(bar(ctl->done[r]), 0, ctl);
    }
  }
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
  __syncthreads();
  if (warp == 0) {
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512));
  }
}

// Joins the splits of an item: one thread per 4 values of a row.
template <int D, int BS, int F>
__global__ void __launch_bounds__(256) attn_prefill_join_kernel(const PrefillArgs pa) {
  const AttnArgs& a = pa.a;
  pdl_wait();
  const int pairs = a.batch * a.heads;
  constexpr int kPerItem = kRowsCta * (D / 4) / 256;  // CTAs per item
  const int item = static_cast<int>(blockIdx.x) / kPerItem;
  const int pair = item % pairs, rt = a.row_tiles - 1 - item / pairs;
  const int h = pair % a.heads, b = pair / a.heads;
  const Span sp = span_of<kRowsCta, TK>(a, b, rt);
  const int e = (static_cast<int>(blockIdx.x) - item * kPerItem) * 256 + threadIdx.x;
  const int row = e / (D / 4), x = (e % (D / 4)) * 4;
  if (row >= sp.rows) return;
  constexpr int64_t kPart = kRowsCta * (D + 2);
  const float* part = a.ws + static_cast<int64_t>(item) * pa.splits * kPart;
  float top = -INFINITY;
#pragma unroll 8
  for (int s = 0; s < pa.splits; ++s) top = fmaxf(top, part[s * kPart + kRowsCta * D + 2 * row]);
  const float ref = top == -INFINITY ? 0.0f : top;
  float sum = 0.0f;
  float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
  for (int s = 0; s < pa.splits; ++s) {
    const float2 ml =
        *reinterpret_cast<const float2*>(part + s * kPart + kRowsCta * D + 2 * row);
    // a part that saw nothing may have left its sums unwritten
    const bool none = ml.x == -INFINITY && ml.y == 0.0f;
    const float f = ex2(ml.x - ref);
    float4 y = *reinterpret_cast<const float4*>(part + s * kPart + row * D + x);
    if (none) y = make_float4(0.f, 0.f, 0.f, 0.f);
    // a NaN sum of a part without a maximum stays NaN
    sum += ml.x == -INFINITY ? ml.y : ml.y * f;
    v.x = fmaf(y.x, f, v.x), v.y = fmaf(y.y, f, v.y);
    v.z = fmaf(y.z, f, v.z), v.w = fmaf(y.w, f, v.w);
  }
  const RowOut<F> out(a, sp, h, sp.r0 + row, top, sum, x == 0);
  const int d = value_at<D, BS>(x);
  out.pair(d, v.x, v.y);
  out.pair(d + 2, v.z, v.w);
}

// ------------------------------------------------------------------- host
// Splits of the tokens where the row tiles alone leave SMs idle: as many as
// fill the SMs once, each at least 4 tiles long.
int splits_for(int64_t items, int64_t span, int num_sms) {
  const int64_t tiles = (span + TK - 1) / TK;
  int64_t s = items > 0 ? num_sms / items : 1;
  if (s > tiles / 4) s = tiles / 4;
  return s < 2 ? 1 : static_cast<int>(s);
}

template <int D, int BS, int F>
cudaError_t launch_t(const PrefillArgs& pa, int64_t items, cudaStream_t s) {
  constexpr int kSmem = Smem<D, F == BNB4_F16>::kOffCtl + static_cast<int>(sizeof(Ctl)) + 1024;
  static_assert(kSmem + (D / BS) * TK * 2 <= 232448, "shared memory budget");
  auto kern = attn_prefill_kernel<D, BS, F>;
  cudaError_t e =
      cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
  if (e != cudaSuccess) return e;
  e = launch_kernel(kern, dim3(static_cast<unsigned>(items * pa.splits)), dim3(kThreads), kSmem, s,
                    programmatic_after_kernel(s), pa);
  if (e != cudaSuccess || pa.splits == 1) return e;
  return launch_kernel(attn_prefill_join_kernel<D, BS, F>,
                       dim3(static_cast<unsigned>(items * (kRowsCta * (D / 4) / 256))), dim3(256),
                       0, s, true, pa);
}

int64_t items_of(const AttnArgs& a, int64_t rows) {
  return static_cast<int64_t>(a.batch) * a.heads * ((rows + kRowsCta - 1) / kRowsCta);
}

}  // namespace

size_t attn_prefill_workspace(const AttnArgs& a, int head_dim, int64_t rows, int64_t span,
                              int num_sms) {
  const int64_t items = items_of(a, rows);
  const int splits = splits_for(items, span, num_sms);
  return splits == 1 ? 0
                     : sizeof(float) * static_cast<size_t>(items) * splits * kRowsCta *
                           (static_cast<size_t>(head_dim) + 2);
}

cudaError_t launch_attn_prefill(AttnArgs& a, const bnb4_kv_cache& c, int64_t rows, int64_t span,
                                int num_sms, cudaStream_t s) {
  PrefillArgs pa;
  a.row_tiles = static_cast<int>((rows + kRowsCta - 1) / kRowsCta);
  const int64_t items = items_of(a, rows);
  pa.splits = splits_for(items, span, num_sms);
  pa.a = a;
#define BNB4_PREFILL(DV, BSV)                                       \
  return c.dtype == BNB4_F16 ? launch_t<DV, BSV, BNB4_F16>(pa, items, s)  \
                             : launch_t<DV, BSV, BNB4_BF16>(pa, items, s);
  if (c.head_dim == 128) {
    if (c.blocksize == 128) { BNB4_PREFILL(128, 128) }
    if (c.blocksize == 64) { BNB4_PREFILL(128, 64) }
    BNB4_PREFILL(128, 32)
  }
  if (c.blocksize == 64) { BNB4_PREFILL(64, 64) }
  BNB4_PREFILL(64, 32)
#undef BNB4_PREFILL
}

}  // namespace bnb4
