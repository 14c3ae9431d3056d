// attn_decode.cu -- attention of a few query rows per sequence over a paged
// 4-bit key/value cache on sm_100a (decode, verified drafts): the tier of
// bnb_attn_4bit for at most 16 rows (queries x grouped heads) per key/value
// head.
//   s_j = scale * sum_b a_k[j, b] * sum_{d in block b} q_d t[k_code[j, d]]
//   o_d = sum_j p_j a_v[j, b(d)] t[v_code[j, d]] / sum_j p_j,  p_j = exp(s_j - m)
// over the tokens j a row sees; t is the 16-entry code table.
//
// Design.
//  * The cache is read once.  A CTA's 12 warps form two groups; a group walks the
//    tiles of 64 (or, for 9 to 16 rows, 32) tokens of one (sequence, key/value head), warp by warp,
//    each with its own running maximum and sums, and joins in shared memory
//    at the end of a segment while the other group's loads keep going.
//  * A warp brings its tiles into its own part of shared memory with bulk
//    copies (one for the codes and one for the scales of 16 tokens, issued
//    by one lane each), keys while the values before them are multiplied and
//    values while the scores form, so neither registers nor address
//    arithmetic of the other lanes are spent on them.
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
//    is multiplied by the constant that brings NF4's fp16 roundings to 3.6e-5 of
//    the scale in the mean square, 8.4e-5 at most, up to 3.1e-4 of a value (FP4 is
//    exact); weights p a_v are scaled by the running power of two of
//    the block's largest a_v, to at most 2^15, so they stay normal fp16 down
//    to 2^-29 of it.  For fp16 outputs, whose last place is finer than those
//    roundings, the weights are split into two fp16 terms and the keys' table
//    entries keep their residue; the values' table stays in one term (a residue
//    would cost a lookup and a product more each), which leaves 1.1 times the
//    error of the output's own rounding for NF4.
//  * Work is split evenly: the tiles of all (sequence, head) pairs form one
//    line that is cut into equal runs, one per CTA; a run's first and last
//    pair may be shared with its neighbours, whose partial results (fp32, in
//    the workspace) a second kernel joins in a fixed order, so results repeat
//    bit for bit.
//
// What bounds it: issued instructions.  16 sequences of 4096
// tokens, 32 heads of 128 (bf16, NF4, blocks of 64): 97 us, 2,940 GB/s of cache
// (44 us at the copy rate); issue slots 55% busy, integer pipe 50%, loads from
// shared memory 48%, DRAM 38%.  A warp issues 1,584 instructions per tile of 64
// tokens, of which the lookups (256 permutes, 256 loads) and the products (64)
// are 576; most of the others are scores, exponentials, weights and transposes,
// where with one row per head 7 of 8 columns are padding.  At 168 registers a
// thread the instantiations with heads of 128 spill: 8 to 180 bytes up to 8 rows,
// 92 to 692 (fp16, NF4, blocks of 32) for 9 to 16.
// Side by side, 12 warps with tiles of 64 tokens
// took 93 us when 16 warps took 99 and 8 warps with tiles of 128 tokens 95.
// 24 ragged sequences with 4 rows per head 64 us, 2 x 131072 tokens 90 us, 12
// sequences with 16 rows (fp16, blocks of 32; weights in two terms) 78 us,
// one sequence of 257 tokens 9.7 us, most of it the launch and three loads in
// a row (lengths, page table, cache).
#include "attn.cuh"
#include "common.cuh"
#include "kvcache.h"
#include "kernels.h"
#include "sm100.cuh"

namespace bnb4 {
namespace {

// ------------------------------------------------------------ primitives
__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                        uint32_t a3, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 "
      "{%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_f16_zero(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                             uint32_t a3, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 "
      "{%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.0f));
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t a) {
  uint32_t d;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
  return d;
}
constexpr uint32_t kTilesAt = 0x1000;   // shared address behind the static arrays
constexpr uint32_t kTableAt = 0x10000;  // and of the pair table

// Address in the table of a code byte's fp16 pair {t[byte >> 4], t[byte &
// 15]}: entry `byte` has 256 bytes, of which the first 128 hold a copy for
// each bank.  lane_base: bytes {4 * lane, 0, 1, 0}; the permute puts byte I of
// w between.
template <int I>
__device__ __forceinline__ uint32_t entry_of(uint32_t w, uint32_t lane_base) {
  uint32_t at;
  asm("prmt.b32 %0, %1, %2, %3;" : "=r"(at) : "r"(w), "r"(lane_base), "n"(0x7604 | (I << 4)));
  return at;
}
template <int OFF>
__device__ __forceinline__ uint32_t pair_at(uint32_t at) {
  uint32_t v;
  asm volatile("ld.shared.u32 %0, [%1+%2];" : "=r"(v) : "r"(at), "n"(OFF));
  return v;
}
template <int I>
__device__ __forceinline__ uint32_t pair_of(uint32_t w, uint32_t lane_base) {
  return pair_at<0>(entry_of<I>(w, lane_base));
}

// KR: the second 128 bytes of an entry hold what the first rounded away.
template <bool KR>
__device__ __forceinline__ void build_table(int qtype, int warp, int warps) {
  const int lane = threadIdx.x & 31;
  const int c = lane & 15;
  const float v = scaled_code(qtype, c);
  const uint32_t h = pack_f16x2(v, 0.0f) & 0xffffu;
  // exact: v is within half an fp16 step of h
  const uint32_t r = pack_f16x2(__fsub_rn(v, half_to_f32<BNB4_F16>(h)), 0.0f) & 0xffffu;
  for (int e = warp; e < 256; e += warps) {
    const uint32_t at = kTableAt + 256u * e + 4u * lane;
    const uint32_t x = __shfl_sync(0xffffffffu, h, e >> 4) | __shfl_sync(0xffffffffu, h, e & 15) << 16;
    asm volatile("st.shared.u32 [%0], %1;" ::"r"(at), "r"(x) : "memory");
    if constexpr (KR) {
      const uint32_t y =
          __shfl_sync(0xffffffffu, r, e >> 4) | __shfl_sync(0xffffffffu, r, e & 15) << 16;
      asm volatile("st.shared.u32 [%0], %1;" ::"r"(at + 128u), "r"(y) : "memory");
    }
  }
}

template <int BYTES>
struct Chunk {  // 4, 8 or 16 bytes of codes
  uint32_t w[BYTES / 4];
  __device__ __forceinline__ void load(uint32_t at) {  // shared address
    if constexpr (BYTES == 16)
      asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];"
                   : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3])
                   : "r"(at));
    else if constexpr (BYTES == 8)
      asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(w[0]), "=r"(w[1]) : "r"(at));
    else
      asm volatile("ld.shared.u32 %0, [%1];" : "=r"(w[0]) : "r"(at));
  }
};

// The NB scales of one token: raw 16-bit patterns, two per word.
template <int NB>
struct Scales {
  uint32_t w[(NB + 1) / 2];
  __device__ __forceinline__ void load(uint32_t at) {
    if constexpr (NB == 1) {
      uint16_t x;
      asm volatile("ld.shared.u16 %0, [%1];" : "=h"(x) : "r"(at));
      w[0] = x;
    } else if constexpr (NB == 2) {
      asm volatile("ld.shared.u32 %0, [%1];" : "=r"(w[0]) : "r"(at));
    } else {
      asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(w[0]), "=r"(w[1]) : "r"(at));
    }
  }
  // finite2: the largest finite pattern in both halves
  __device__ __forceinline__ bool not_finite(uint32_t finite2) const {
    uint32_t x = w[0];
    if constexpr (NB == 4) x = __vmaxu2(x, w[1]);
    return __vmaxu2(x, finite2) != finite2;
  }
  template <int F>
  __device__ __forceinline__ float at(int b) const {
    const uint32_t x = w[b / 2];
    if constexpr (F == BNB4_BF16)
      return (b & 1) ? bf16_hi(x) : bf16_lo(x);
    else
      return half_to_f32<F>((b & 1) ? x >> 16 : x & 0xffffu);
  }
};

__device__ __forceinline__ void copy_to_shared(uint32_t dst, const void* src, uint32_t bytes,
                                               uint32_t bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::
          "r"(dst),
      "l"(src), "r"(bytes), "r"(bar)
      : "memory");
}
__device__ __forceinline__ void group_sync(int group, int threads) {
  asm volatile("bar.sync %0, %1;" ::"r"(group + 1), "r"(threads) : "memory");
}

// ------------------------------------------------------------- the kernel
// D, BS: head dimension and block size.  F: the 16-bit type.  NT: 8-row
// groups of the row tile.  KR: the keys' table entries keep their rounding
// residue in a second fp16 (fp16 caches with the NF4 table).
template <int D, int BS, int F, int NT, bool KR>
struct Shape {
  static constexpr int NS = NT == 1 ? 4 : 2;           // 16-token sub-tiles per tile
  static constexpr int ST = NT == 1 ? 1 : 2;           // tiles in flight per warp
  static constexpr int W = 12;                         // warps
  static constexpr int GW = W / 2;                     // warps per group
  static constexpr int RT = 8 * NT, TILE = 16 * NS, NB = D / BS, KS = D / 16;
  static constexpr int kCodes = TILE * D / 2, kScales = TILE * NB * 2;
  static constexpr int kStage = kCodes + kScales;      // one tile of keys, or of values
  static constexpr int kWarp = 2 * ST * kStage;
  // joining: up to kGive of a group's warps hand over at a time, one 128-byte
  // piece per accumulator register
  static constexpr int kGive = NT == 1 ? GW / 2 : 2;
  static constexpr int kPieces = kGive * KS * NT * 4;
  // where the table's entries use only half of their 256 bytes the pieces lie
  // in the other half, else behind the warps' tiles
  static constexpr bool kGaps = !KR && 2 * kPieces <= 256;
  // shared addresses: the first warps' tiles below the table, the others' above
  static constexpr int kBelow =
      static_cast<int>(kTableAt - kTilesAt) / kWarp < W ? static_cast<int>(kTableAt - kTilesAt) / kWarp : W;
  static constexpr uint32_t kAbove = kTableAt + 0x10000;
  static constexpr uint32_t kJoin = kAbove + (W - kBelow) * kWarp;
  static constexpr uint32_t kEnd = kJoin + (kGaps ? 0 : 2 * kPieces * 128);
  __device__ static __forceinline__ uint32_t tiles(int warp) {
    return warp < kBelow ? kTilesAt + static_cast<uint32_t>(warp) * kWarp
                         : kAbove + static_cast<uint32_t>(warp - kBelow) * kWarp;
  }
  __device__ static __forceinline__ uint32_t piece(int group, int i) {
    const uint32_t p = static_cast<uint32_t>(group * kPieces + i);
    return kGaps ? kTableAt + 128u + 256u * p : kJoin + 128u * p;
  }
};

struct Ctl {  // the fields that a bounded wait looks at
  uint64_t wait_limit_ns;
  int abort;
};

template <int D, int BS, int F, int NT, bool KR>
__global__ void __launch_bounds__(Shape<D, BS, F, NT, KR>::W * 32, 1)
    attn_decode_kernel(const AttnArgs a) {
  using S = Shape<D, BS, F, NT, KR>;
  constexpr int NS = S::NS, ST = S::ST, W = S::W, GW = S::GW, RT = S::RT, TILE = S::TILE;
  constexpr int NB = S::NB, KS = S::KS;
  constexpr int SW = BS / 8;  // values of a block per strip
  constexpr bool kSplitP = F == BNB4_F16;
  constexpr uint32_t kInf = F == BNB4_BF16 ? 0x7f80u : 0x7c00u;
  extern __shared__ uint8_t smem_raw[];
  __shared__ uint64_t bars[W][2 * ST];
  __shared__ Ctl ctl;
  __shared__ float sm_m[W][RT], sm_l[W][RT], sm_max[2][RT], sm_sum[2][RT];
  __shared__ int sm_item[2][4];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int grp = warp / GW, gw = warp - grp * GW;
  const int g = lane >> 2, t = lane & 3;
  const uint32_t lane_base = kTableAt | (4u * lane);
  // the fixed places must lie behind the static arrays and inside the dynamic
  // ones (the launch asks for enough); refused here if they do not
  if (smem_u32(smem_raw) > kTilesAt || smem_u32(bars) + sizeof(bars) > kTilesAt ||
      smem_u32(&ctl) + sizeof(ctl) > kTilesAt || smem_u32(sm_m) + sizeof(sm_m) > kTilesAt ||
      smem_u32(sm_l) + sizeof(sm_l) > kTilesAt || smem_u32(sm_max) + sizeof(sm_max) > kTilesAt ||
      smem_u32(sm_sum) + sizeof(sm_sum) > kTilesAt || smem_u32(sm_item) + sizeof(sm_item) > kTilesAt) {
    if (threadIdx.x == 0) atomicExch(a.err, 1);
    return;
  }
  pdl_trigger();
  if (lane == 0) {
#pragma unroll
    for (int i = 0; i < 2 * ST; ++i) mbar_init(smem_u32(&bars[warp][i]), 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (threadIdx.x == 0) {
    ctl.wait_limit_ns = a.wait_limit_ns;
    ctl.abort = 0;
  }
  // the table is built by the warps that do not look for their group's run below
  if (gw != 0) build_table<KR>(a.qtype, warp - 1 - grp, W - 2);
  pdl_wait();

  // -------- this group's run of the line of tiles, or its items in turn
  const int run = static_cast<int>(blockIdx.x) * 2 + grp, runs = 2 * static_cast<int>(gridDim.x);
  if (a.split && gw == 0) {
    int64_t total = 0;
    for (int b0 = 0; b0 < a.batch; b0 += 32) {
      const int i = b0 + lane;
      total += i < a.batch ? static_cast<int64_t>(span_of<RT, TILE>(a, i, 0).tiles) : 0;
    }
    total = warp_sum(total) * a.heads;
    const int64_t per = (total + runs - 1) / runs;
    const int64_t u0 = per * run;
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
      sm_item[grp][0] = fb;
      sm_item[grp][1] = fh;
      sm_item[grp][2] = ft;
      sm_item[grp][3] = static_cast<int>(mine);
    }
  }
  __syncthreads();
  // this warp's tiles: ST of keys, then ST of values
  const uint32_t my_k = S::tiles(warp);
  const uint32_t my_v = my_k + ST * S::kStage;
  // a lane's copies: where in a stage, how many bytes, from which array
  const int copy_u = lane >> 1;
  const uint32_t copy_at =
      lane & 1 ? S::kCodes + copy_u * (S::kScales / NS) : copy_u * (S::kCodes / NS);
  const uint32_t copy_bytes = lane & 1 ? S::kScales / NS : S::kCodes / NS;
  const int copy_row = lane & 1 ? 2 * NB : D / 2;
  const uint8_t* copy_k = lane & 1 ? reinterpret_cast<const uint8_t*>(a.k_absmax) : a.k_codes;
  const uint8_t* copy_v = lane & 1 ? reinterpret_cast<const uint8_t*>(a.v_absmax) : a.v_codes;
  uint32_t put = 0, got = 0;  // tiles issued and consumed; slot = count % ST
  bool ok_all = true;         // no wait of this warp gave up

  // The group's segments: the pair (b, h) and its tiles tile0 .. tile1 - 1.
  struct Seg {
    int b, h, tile0, tile1;
    Span sp;
  };
  int left = a.split ? sm_item[grp][3] : 0;  // tiles left of the run
  int64_t item = run;
  const int64_t items = static_cast<int64_t>(a.batch) * a.heads;
  // the next segment from (b, h, tile0) on; false: there is none
  auto find = [&](Seg& g2) {
    if (a.split) {
      while (left > 0 && g2.b < a.batch) {
        g2.sp = span_of<RT, TILE>(a, g2.b, 0);
        if (g2.sp.rows > 0) {
          g2.tile1 = g2.sp.tiles - g2.tile0 <= left ? g2.sp.tiles : g2.tile0 + left;
          left -= g2.tile1 - g2.tile0;
          return true;
        }
        ++g2.b, g2.h = 0, g2.tile0 = 0;  // holds no tiles
      }
    } else {
      for (; item < items; item += runs) {
        g2.h = static_cast<int>(item % a.heads);
        g2.b = static_cast<int>(item / a.heads);
        g2.sp = span_of<RT, TILE>(a, g2.b, 0);
        if (g2.sp.rows > 0) {
          g2.tile0 = 0, g2.tile1 = g2.sp.tiles;
          item += runs;
          return true;
        }
      }
    }
    return false;
  };

  // A tile's copies: lane 2 u brings sub-tile u's codes, lane 2 u + 1 its
  // scales.  The page entry of the lane's sub-tile of tile i (-1: no cached
  // token) is read a tile ahead of its use.
  auto page_of = [&](const Seg& w, int i) {
    const int j = w.sp.base + i * TILE + 16 * (lane >> 1);
    return lane < 2 * NS && i < w.tile1 && j < w.sp.end
               ? __ldg(a.block_table + static_cast<int64_t>(w.b) * a.bt_stride +
                       a.page.div(static_cast<uint32_t>(j)))
               : -1;
  };
  auto row_of = [&](const Seg& w, int i, int entry) {  // the sub-tile's first cache row, or -1
    const uint32_t j = static_cast<uint32_t>(w.sp.base + i * TILE + 16 * (lane >> 1));
    const uint32_t in = j - a.page.div(j) * a.page.d;
    return entry >= 0 && entry < a.num_pages
               ? (static_cast<int64_t>(entry) * a.heads + w.h) * a.page.d + in
               : static_cast<int64_t>(-1);
  };
  // into slot n % ST; returns bit 2 u for each sub-tile u that is there.  hold: the
  // lane's copy is counted but not made (failure-detection diagnostic).
  auto issue = [&](int64_t row, uint32_t n, bool values, bool hold = false) {
    const uint32_t at = (values ? my_v : my_k) + (n % ST) * S::kStage + copy_at;
    const uint32_t bar = smem_u32(&bars[warp][(values ? ST : 0) + n % ST]);
    const unsigned have = __ballot_sync(0xffffffffu, row >= 0) & 0x55555555u;
    if (lane == 0)
      mbar_arrive_expect_tx(bar, __popc(have) * (S::kCodes / NS + S::kScales / NS));
    __syncwarp();  // also orders the slot's last reads before the copies
    if (row >= 0 && !hold)
      copy_to_shared(at, (values ? copy_v : copy_k) + row * copy_row, copy_bytes, bar);
    return have;
  };
  auto wait = [&](uint32_t n, bool values) {
    const uint32_t bar = smem_u32(&bars[warp][(values ? ST : 0) + n % ST]);
    // Every lane asks for itself, and one may see the phase complete where another
    // sees that the CTA gives up: the warp decides as one, since all that it does
    // next (votes, shuffles, products) takes all its lanes.
    if (!__all_sync(0xffffffffu, wait_bounded(bar, (n / ST) & 1, &ctl, a.err))) ok_all = false;
  };

  // Starts a segment: its first tiles are on their way, and its rows of q (as B
  // operand of every k-step: rows g and g + 8) are being read -- with 16 rows
  // only later, for want of registers while the segment before is joined.
  constexpr uint32_t kAll = 0x55u & ((1u << 2 * NS) - 1);
  unsigned have = 0;  // sub-tiles present, 2 NS bits per tile in flight, oldest lowest
  int entry_next = -1;
  uint32_t raw[NT][KS][2];
  auto read_q = [&](const Seg& w) {
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const bool real = 8 * n + g < w.sp.rows;
      const int r = real ? w.sp.r0 + 8 * n + g : 0;
      const int i = r / a.group, hh = r - i * a.group;
      const uint16_t* src = a.q + (static_cast<int64_t>(w.sp.q0) + i) * a.q_ts +
                            (static_cast<int64_t>(w.h) * a.group + hh) * a.q_hs;
#pragma unroll
      for (int s = 0; s < KS; ++s)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          // stored place of the pair, and the dimension it holds
          const int p = t * (D / 4) + 4 * s + 2 * e;
          const int strip = p / (D / 8), x = p % (D / 8);
          const int d = (x / SW) * BS + strip * SW + x % SW;
          raw[n][s][e] = real ? __ldg(reinterpret_cast<const uint32_t*>(src + d)) : 0u;
        }
    }
  };
  auto start = [&](const Seg& w) {
    int entry[ST + 1];
#pragma unroll
    for (int x = 0; x < ST + 1; ++x) entry[x] = page_of(w, w.tile0 + gw + x * GW);
    if constexpr (NT == 1) read_q(w);
    have = 0;
#pragma unroll
    for (int x = 0; x < ST; ++x) {
      const int i = w.tile0 + gw + x * GW;
      if (i < w.tile1 && ok_all) {  // after a failed wait nothing more is issued, but
                                    // the group's barriers below are still met
        const int64_t row = row_of(w, i, entry[x]);
        have |= issue(row, put, false, a.withhold && blockIdx.x == 0 && threadIdx.x == 1)
                << (2 * NS * x);
        issue(row, put, true);
        ++put;
      }
    }
    entry_next = entry[ST];
  };

  Seg cur;
  cur.b = cur.h = cur.tile0 = 0;
  if (a.split) cur.b = sm_item[grp][0], cur.h = sm_item[grp][1], cur.tile0 = sm_item[grp][2];
  bool more_segs = find(cur);
  if (more_segs) start(cur);
  while (more_segs) {  // uniform over the group
    const Span sp = cur.sp;
    const int h = cur.h, tile0 = cur.tile0, tile1 = cur.tile1;
    if constexpr (NT > 1) read_q(cur);
    uint32_t qf[NT][KS][2];
    float qs[NT][2];  // per column 2 t, 2 t + 1: score in log2 units = sum of products * qs
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      uint32_t top = 0;
#pragma unroll
      for (int s = 0; s < KS; ++s)
#pragma unroll
        for (int e = 0; e < 2; ++e)
          top = max(top, max(raw[n][s][e] & 0x7fffu, (raw[n][s][e] >> 16) & 0x7fffu));
      top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
      top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
      float mul = a.scale_log2;
      // a row with an infinite or NaN entry is NaN as a whole, so every score of a
      // token that it sees is; `mul` stays finite, so that a token that it does not
      // see keeps its weight of zero
      const uint32_t poison = top >= kInf ? 0x7fff7fffu : 0u;
#pragma unroll
      for (int s = 0; s < KS; ++s) raw[n][s][0] |= poison, raw[n][s][1] |= poison;
      if constexpr (F == BNB4_BF16) {
        int e = static_cast<int>(top >> 7) - 127;  // exponent of the row's largest
        e = e < -100 ? -100 : e;
        const float f = pow2(14 - e);
        mul *= pow2(e - 14);
#pragma unroll
        for (int s = 0; s < KS; ++s)
#pragma unroll
          for (int x = 0; x < 2; ++x)
            qf[n][s][x] = pack_f16x2(bf16_lo(raw[n][s][x]) * f, bf16_hi(raw[n][s][x]) * f);
      } else {
#pragma unroll
        for (int s = 0; s < KS; ++s) qf[n][s][0] = raw[n][s][0], qf[n][s][1] = raw[n][s][1];
      }
      mul *= a.qtype == kQtNF4 ? 1.0f / kNf4Scale : 1.0f / kFp4Scale;
      // columns 2 t and 2 t + 1 are rows held by lanes 4 (2 t) and 4 (2 t + 1)
      qs[n][0] = __shfl_sync(0xffffffffu, mul, 8 * t);
      qs[n][1] = __shfl_sync(0xffffffffu, mul, 8 * t + 4);
    }
    // tokens every row sees: tiles inside need no mask
    const int pos0 = sp.first + sp.r0 / a.group;
    const int all_hi = a.causal && pos0 < sp.len ? pos0 : sp.len - 1;
    const int all_lo = a.window > 0 ? sp.first + (sp.r0 + sp.rows - 1) / a.group - a.window + 1 : 0;

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

    // MMA row r of a sub-tile is its token r ^ (r >> 1 & 1): neighbouring rows
    // differ in parity (keys), and so do rows 2 t and 2 t + 2 (values), which
    // spreads their 64-byte rows over the banks
    const int tok_g = g ^ ((g >> 1) & 1);

    for (int i = tile0 + gw; i < tile1 && ok_all; i += GW) {
      const uint32_t ok = have & kAll;
      have >>= 2 * NS;
      const uint32_t kb = my_k + (got % ST) * S::kStage, vb = my_v + (got % ST) * S::kStage;
      wait(got, false);
      // ------------------------------------------------ scores
      float s[NS][NT][4];
      uint32_t kmax = 0;  // largest patterns of the key scales, in both halves
#pragma unroll
      for (int u = 0; u < NS; ++u) {
        Chunk<D / 8> k0, k1;
        k0.load(kb + (16 * u + tok_g) * (D / 2) + t * (D / 8));
        k1.load(kb + (16 * u + tok_g + 8) * (D / 2) + t * (D / 8));
        Scales<NB> s0, s1;
        s0.load(kb + S::kCodes + (16 * u + tok_g) * (2 * NB));
        s1.load(kb + S::kCodes + (16 * u + tok_g + 8) * (2 * NB));
#pragma unroll
        for (int y = 0; y < (NB + 1) / 2; ++y) kmax = __vmaxu2(kmax, __vmaxu2(s0.w[y], s1.w[y]));
#pragma unroll
        for (int blk = 0; blk < NB; ++blk) {
          float acc[NT][4];
          bool first = true;
#pragma unroll
          for (int st = 0; st < KS; ++st) {
            // k-step st: bytes 2 st and 2 st + 1 of the lane's two strips
            if (((st % (KS / 2)) * 4) / SW != blk) continue;
            const uint32_t w0 = k0.w[st / 2], w1 = k1.w[st / 2];
            uint32_t x0, x1, x2, x3;  // table addresses
            if (st % 2 == 0) {
              x0 = entry_of<0>(w0, lane_base), x1 = entry_of<0>(w1, lane_base);
              x2 = entry_of<1>(w0, lane_base), x3 = entry_of<1>(w1, lane_base);
            } else {
              x0 = entry_of<2>(w0, lane_base), x1 = entry_of<2>(w1, lane_base);
              x2 = entry_of<3>(w0, lane_base), x3 = entry_of<3>(w1, lane_base);
            }
            const uint32_t a0 = pair_at<0>(x0), a1 = pair_at<0>(x1), a2 = pair_at<0>(x2),
                           a3 = pair_at<0>(x3);
#pragma unroll
            for (int n = 0; n < NT; ++n) {
              if (first)
                mma_f16_zero(acc[n], a0, a1, a2, a3, qf[n][st][0], qf[n][st][1]);
              else
                mma_f16(acc[n], a0, a1, a2, a3, qf[n][st][0], qf[n][st][1]);
            }
            if constexpr (KR) {
              const uint32_t r0 = pair_at<128>(x0), r1 = pair_at<128>(x1), r2 = pair_at<128>(x2),
                             r3 = pair_at<128>(x3);
#pragma unroll
              for (int n = 0; n < NT; ++n)
                mma_f16(acc[n], r0, r1, r2, r3, qf[n][st][0], qf[n][st][1]);
            }
            first = false;
          }
          const float f0 = s0.template at<F>(blk), f1 = s1.template at<F>(blk);
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            s[u][n][0] = blk ? fmaf(acc[n][0], f0, s[u][n][0]) : acc[n][0] * f0;
            s[u][n][1] = blk ? fmaf(acc[n][1], f0, s[u][n][1]) : acc[n][1] * f0;
            s[u][n][2] = blk ? fmaf(acc[n][2], f1, s[u][n][2]) : acc[n][2] * f1;
            s[u][n][3] = blk ? fmaf(acc[n][3], f1, s[u][n][3]) : acc[n][3] * f1;
          }
        }
      }
      // an infinite scale makes every product infinite or NaN: a token with a
      // scale that is not finite has a NaN score
      constexpr uint32_t kFinite2 = (kInf - 1) * 0x10001u;
      if (__any_sync(0xffffffffu, __vmaxu2(kmax, kFinite2) != kFinite2)) {
#pragma unroll
        for (int u = 0; u < NS; ++u)
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            Scales<NB> sc;
            sc.load(kb + S::kCodes + (16 * u + tok_g + 8 * x) * (2 * NB));
            if (sc.not_finite(kFinite2))
#pragma unroll
              for (int n = 0; n < NT; ++n)
                s[u][n][2 * x] = s[u][n][2 * x + 1] = __int_as_float(0x7fffffff);
          }
      }
      // the next tile's keys are on their way while this one's weights form
      const bool more = i + ST * GW < tile1;
      int64_t row_next = -1;
      if (more && ok_all) {
        row_next = row_of(cur, i + ST * GW, entry_next);
        have |= issue(row_next, put, false) << (2 * NS * (ST - 1));
      }
      entry_next = page_of(cur, i + (ST + 1) * GW);

      const int j0 = sp.base + i * TILE;
      const bool masked = ok != kAll || j0 < all_lo || j0 + TILE - 1 > all_hi;  // warp-uniform
      if (masked) {
        asm volatile("" ::: "memory");  // a branch, not selects on every tile
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            // last (inclusive) and first token that column 2 t + c sees
            const int r = 8 * n + 2 * t + c;
            const int pos = sp.first + (sp.r0 + r) / a.group;
            const int hi = r >= sp.rows ? -1 : a.causal && pos < sp.len ? pos : sp.len - 1;
            const int lo = a.window > 0 ? pos - a.window + 1 : 0;
#pragma unroll
            for (int u = 0; u < NS; ++u)
#pragma unroll
              for (int x = 0; x < 2; ++x) {
                const int j = j0 + 16 * u + tok_g + 8 * x;
                if (!((ok >> (2 * u)) & 1u) || j > hi || j < lo) s[u][n][c + 2 * x] = -INFINITY;
              }
          }
      }
      float top[NT][2];
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          float x = -INFINITY;
#pragma unroll
          for (int u = 0; u < NS; ++u) x = fmaxf(x, fmaxf(s[u][n][c], s[u][n][c + 2]));
#pragma unroll
          for (int y = 4; y <= 16; y <<= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, y));
          top[n][c] = fmaxf(m[n][c], __fmul_rn(x, qs[n][c]));  // qs > 0; drops NaN
        }
      wait(got, true);
      Scales<NB> vs[NS][2];
      uint32_t vmax[(NB + 1) / 2] = {};
#pragma unroll
      for (int u = 0; u < NS; ++u)
#pragma unroll
        for (int x = 0; x < 2; ++x) vs[u][x].load(vb + S::kCodes + (16 * u + tok_g + 8 * x) * (2 * NB));
      if (masked) {  // scales of tokens that no row sees may be anything
        asm volatile("" ::: "memory");
#pragma unroll
        for (int u = 0; u < NS; ++u)
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            const int j = j0 + 16 * u + tok_g + 8 * x;
            if (!((ok >> (2 * u)) & 1u) || j >= sp.end || j < sp.lo)
#pragma unroll
              for (int y = 0; y < (NB + 1) / 2; ++y) vs[u][x].w[y] = 0u;
          }
      }
#pragma unroll
      for (int u = 0; u < NS; ++u)
#pragma unroll
        for (int y = 0; y < (NB + 1) / 2; ++y)
          vmax[y] = __vmaxu2(vmax[y], __vmaxu2(vs[u][0].w[y], vs[u][1].w[y]));
      {
        uint32_t x = vmax[0];
        if constexpr (NB == 4) x = __vmaxu2(x, vmax[1]);
        if (__any_sync(0xffffffffu, __vmaxu2(x, kFinite2) != kFinite2)) {
          // a value with a scale that is not finite makes the rows that see its
          // token NaN, and counts as zero for the others
#pragma unroll
          for (int y = 0; y < (NB + 1) / 2; ++y) vmax[y] = 0;
#pragma unroll
          for (int u = 0; u < NS; ++u)
#pragma unroll
            for (int y = 0; y < 2; ++y) {
              if (vs[u][y].not_finite(kFinite2)) {
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                  for (int c = 0; c < 2; ++c)
                    if (s[u][n][2 * y + c] != -INFINITY) l[n][c] = __int_as_float(0x7fffffff);
#pragma unroll
                for (int z = 0; z < (NB + 1) / 2; ++z) vs[u][y].w[z] = 0u;
              }
#pragma unroll
              for (int z = 0; z < (NB + 1) / 2; ++z) vmax[z] = __vmaxu2(vmax[z], vs[u][y].w[z]);
            }
        }
      }
      // running exponents of the value scales, and the factor that brings a
      // weight times its scale to at most 2^15
      float vn[NB], vgrow[NB];
      bool up = false;
#pragma unroll
      for (int blk = 0; blk < NB; ++blk) {
        const uint32_t w = vmax[blk / 2];
        const uint32_t x = __reduce_max_sync(0xffffffffu, (blk & 1) ? w >> 16 : w & 0xffffu);
        const int e =
            F == BNB4_BF16 ? static_cast<int>(x >> 7) - 127 : static_cast<int>(x >> 10) - 15;
        vgrow[blk] = 1.0f;
        if (e > ve[blk]) {
          const int d = ve[blk] - e;
          vgrow[blk] = d < -126 ? 0.0f : pow2(d);
          ve[blk] = e;
          up = true;
        }
        vn[blk] = pow2(14 - ve[blk]);
      }
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
      float ref[NT][2];
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int c = 0; c < 2; ++c) ref[n][c] = m[n][c] == -INFINITY ? 0.0f : m[n][c];
      // Scores to the weights' exponents.  Where they are so large that half a step
      // of theirs counts, the product is rounded as the maximum's was before the
      // maximum is taken off, so that the largest weight is one (an fma would
      // leave that half step).
      bool far = false;
#pragma unroll
      for (int n = 0; n < NT; ++n) far = far || fmaxf(fabsf(ref[n][0]), fabsf(ref[n][1])) > kFarScore;
      if (__any_sync(0xffffffffu, far)) {
        asm volatile("" ::: "memory");
#pragma unroll
        for (int u = 0; u < NS; ++u)
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int c = 0; c < 4; ++c)
              s[u][n][c] = __fsub_rn(__fmul_rn(s[u][n][c], qs[n][c & 1]), ref[n][c & 1]);
      } else {
#pragma unroll
        for (int u = 0; u < NS; ++u)
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int c = 0; c < 4; ++c)
              s[u][n][c] = fmaf(s[u][n][c], qs[n][c & 1], -ref[n][c & 1]);
      }
      // ------------------------------------------------ weights and values
#pragma unroll
      for (int u = 0; u < NS; ++u) {
        Chunk<D / 16> v[4];  // the lane's strip of tokens 2 t, 2 t + 1 and 8 more of each
#pragma unroll
        for (int c = 0; c < 4; ++c)
          v[c].load(vb + (16 * u + ((2 * t + (c & 1)) ^ (t & 1)) + 8 * (c >> 1)) * (D / 2) +
                    g * (D / 16));
        uint32_t pb[NB][NT][2], pl[NB][NT][2];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          float p[4];
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            p[c] = ex2(s[u][n][c]);
            l[n][c & 1] += p[c];
          }
#pragma unroll
          for (int blk = 0; blk < NB; ++blk)
#pragma unroll
            for (int x = 0; x < 2; ++x) {
              const float av = vs[u][x].template at<F>(blk) * vn[blk];
              const float y0 = p[2 * x] * av, y1 = p[2 * x + 1] * av;
              const uint32_t hi = pack_f16x2(y0, y1);
              pb[blk][n][x] = transpose8x8(hi);
              if constexpr (kSplitP)
                pl[blk][n][x] = transpose8x8(pack_f16x2(
                    y0 - half_to_f32<BNB4_F16>(hi & 0xffffu), y1 - half_to_f32<BNB4_F16>(hi >> 16)));
            }
        }
#pragma unroll
        for (int wd = 0; wd < D / 64; ++wd) {
          // word wd of the strip for the 4 tokens: bytes of the codes of two
          // tokens (even values; odd values)
          const uint32_t w0 = v[0].w[wd], w1 = v[1].w[wd], w2 = v[2].w[wd], w3 = v[3].w[wd];
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
      if (!ok_all) break;  // what is in flight is waited for below
      ++got;
      if (more) {
        issue(row_next, put, true);
        ++put;
      }
    }
    // ---------------------------------------------------- join the warps
    // the next segment's first tiles are on their way meanwhile
    if (a.split) {
      cur.tile0 = 0;
      if (++cur.h == a.heads) cur.h = 0, ++cur.b;
    }
    more_segs = find(cur);
    if (more_segs) start(cur);

    const int busy = tile1 - tile0 < GW ? tile1 - tile0 : GW;  // warps with a tile
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
    group_sync(grp, GW * 32);
    if (gw == 0 && lane < RT) {
      float top = -INFINITY;
      for (int w = 0; w < busy; ++w) top = fmaxf(top, sm_m[grp * GW + w][lane]);
      const float r = top == -INFINITY ? 0.0f : top;
      float sum = 0.0f;
      for (int w = 0; w < busy; ++w) sum += sm_l[grp * GW + w][lane] * ex2(sm_m[grp * GW + w][lane] - r);
      sm_max[grp][lane] = top;
      sm_sum[grp][lane] = sum;
    }
    const float cinv = a.qtype == kQtNF4 ? 1.0f / kNf4Scale : 1.0f / kFp4Scale;
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        // every warp finds the common maximum for its own columns
        float top = -INFINITY;
        for (int w = 0; w < busy; ++w) top = fmaxf(top, sm_m[grp * GW + w][8 * n + 2 * t + c]);
        const float f = ex2(m[n][c] - (top == -INFINITY ? 0.0f : top)) * cinv;
#pragma unroll
        for (int x = 0; x < KS; ++x) {
          const float back = pow2(ve[(2 * x) / SW] - 14);
          o[x][n][c] = o[x][n][c] * f * back;
          o[x][n][c + 2] = o[x][n][c + 2] * f * back;
        }
      }
    // The warps behind the first H hand their sums over to those (H at a time),
    // these put theirs down, and all warps add them up, a share of the values
    // each: a fixed order.
    constexpr int H = S::kGive;
    auto put_down = [&](int slot) {
#pragma unroll
      for (int x = 0; x < KS; ++x)
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int c = 0; c < 4; ++c)
            asm volatile("st.shared.f32 [%0], %1;" ::"r"(
                             S::piece(grp, (slot * KS + x) * NT * 4 + n * 4 + c) + 4u * lane),
                         "f"(o[x][n][c])
                         : "memory");
    };
    auto piece_at = [&](int slot, int x, int n, int c) {
      float y;
      asm volatile("ld.shared.f32 %0, [%1];"
                   : "=f"(y)
                   : "r"(S::piece(grp, (slot * KS + x) * NT * 4 + n * 4 + c) + 4u * lane));
      return y;
    };
#pragma unroll 1
    for (int first = H; first < busy; first += H) {
      if (first > H) group_sync(grp, GW * 32);  // the slots have been read
      if (gw >= first && gw < first + H && gw < busy) put_down(gw - first);
      group_sync(grp, GW * 32);
      if (gw < H && first + gw < busy) {
#pragma unroll
        for (int x = 0; x < KS; ++x)
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int c = 0; c < 4; ++c) o[x][n][c] += piece_at(gw, x, n, c);
      }
    }
    if (gw < H && gw < busy) put_down(gw);  // its own slot, which it read last
    group_sync(grp, GW * 32);
    const bool whole = tile0 == 0 && tile1 == sp.tiles;
    // partial results: slot 0 continues the run before, slot 1 goes on in the next
    float* part = a.ws + (static_cast<int64_t>(run) * 2 + (tile0 == 0 ? 1 : 0)) *
                             (RT * D + 2 * RT);
    const int slots = busy < H ? busy : H;
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const int r = 8 * n + 2 * t + c;
        if (r < sp.rows) {
          const float top = sm_max[grp][r], sum = sm_sum[grp][r];
          const RowOut<F> out(a, sp, h, sp.r0 + r, top, sum, whole && gw == 0 && g == 0);
          if (!whole && gw == 0 && g == 0) {
            part[RT * D + r] = top;
            part[RT * D + RT + r] = sum;
          }
          for (int x = gw; x < KS; x += GW) {
            float y0 = piece_at(0, x, n, c), y1 = piece_at(0, x, n, c + 2);
            for (int w = 1; w < slots; ++w) y0 += piece_at(w, x, n, c), y1 += piece_at(w, x, n, c + 2);
            const int d = (2 * x / SW) * BS + g * SW + (2 * x) % SW;  // two values of a block
            if (whole)
              out.pair(d, y0, y1);
            else
              *reinterpret_cast<float2*>(part + r * D + d) = make_float2(y0, y1);
          }
        }
      }
    group_sync(grp, GW * 32);  // the shared arrays are free for the next segment
  }
  // a wait that gave up: copies in flight (of tile `put` the keys at most) land
  // before the CTA ends
  if (!ok_all)
    for (uint32_t n = got; n < put + 1; ++n)
      for (int v = 0; v < 2; ++v)
        wait_drain(smem_u32(&bars[warp][(v ? ST : 0) + n % ST]), (n / ST) & 1, &ctl);
}

// Joins the partial results of the pairs that several runs share: CTA i takes
// the pair that begins in run i and goes on in run i + 1.
// A pair may be shared by all runs (few pairs, a long context), so the parts are
// spread over the threads, and weighted first.
constexpr int kMaxRuns = 320;  // bound of the runs, hence of the workspace
constexpr int kJoinThreads = 1024;

template <int D, int F, int NT, int TILE>
__global__ void __launch_bounds__(kJoinThreads) attn_join_kernel(const AttnArgs a) {
  constexpr int RT = 8 * NT;
  __shared__ int sm_item[5];
  __shared__ float sm_f[kMaxRuns * RT], sm_top[RT], sm_sum[RT];
  __shared__ float4 sm_v[kJoinThreads];
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
  const int n = last - static_cast<int>(run) + 1, rows = sp.rows;
  // part x: this run's second slot, then the first one of the runs behind it
  auto part_at = [&](int x) { return a.ws + (2 * (run + x) + (x == 0 ? 1 : 0)) * kPart; };
  for (int e = threadIdx.x; e < n * rows; e += kJoinThreads)
    sm_f[e] = part_at(e / rows)[RT * D + e % rows];
  __syncthreads();
  const int warp = threadIdx.x >> 5;
  if (warp < rows) {  // a row per warp: the maximum, then weights relative to it
    float top = -INFINITY;
    for (int x = lane; x < n; x += 32) top = fmaxf(top, sm_f[x * rows + warp]);
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    const float ref = top == -INFINITY ? 0.0f : top;
    float sum = 0.0f;
    for (int x = lane; x < n; x += 32) {
      const float m = sm_f[x * rows + warp], l = part_at(x)[RT * D + RT + warp];
      const float f = ex2(m - ref);
      sm_f[x * rows + warp] = f;
      sum += m == -INFINITY ? l : l * f;  // a NaN sum without a maximum stays NaN
    }
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if (lane == 0) sm_top[warp] = top, sm_sum[warp] = sum;
  }
  __syncthreads();
  const int values = rows * (D / 4), groups = kJoinThreads / values;
  const int grp = threadIdx.x / values, e = threadIdx.x - grp * values;
  const int r = e / (D / 4), d = (e % (D / 4)) * 4;
  float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
  if (grp < groups) {
#pragma unroll 4
    for (int x = grp; x < n; x += groups) {
      const float f = sm_f[x * rows + r];
      const float4 y = *reinterpret_cast<const float4*>(part_at(x) + r * D + d);
      v.x = fmaf(y.x, f, v.x), v.y = fmaf(y.y, f, v.y);
      v.z = fmaf(y.z, f, v.z), v.w = fmaf(y.w, f, v.w);
    }
    sm_v[threadIdx.x] = v;
  }
  __syncthreads();
  if (grp == 0) {
    for (int x = 1; x < groups; ++x) {
      const float4 y = sm_v[x * values + e];
      v.x += y.x, v.y += y.y, v.z += y.z, v.w += y.w;
    }
    const RowOut<F> out(a, sp, h, r, sm_top[r], sm_sum[r], d == 0);
    out.pair(d, v.x, v.y);
    out.pair(d + 2, v.z, v.w);
  }
}

// ------------------------------------------------------------------- host
// Whole pairs in turn where no pair has more than a tile per warp of a group
// (a cut would only add the join), else the line of tiles cut into equal runs.
template <int F, int NT, bool KR>
constexpr int64_t unsplit_span() {
  using S = Shape<128, 128, F, NT, KR>;  // the same for every head and block size
  return S::TILE * S::GW;
}

template <int D, int BS, int F, int NT, bool KR>
cudaError_t launch_t(AttnArgs& a, int64_t span, int num_sms, cudaStream_t s) {
  using S = Shape<D, BS, F, NT, KR>;
  // The arrays' shared addresses are fixed: everything from the first byte of
  // shared memory to kEnd must be there (static and reserved bytes come off).
  constexpr int kSmem = static_cast<int>(S::kEnd);
  static_assert(kSmem + 4096 <= 232448, "shared memory budget");
  a.split = span > unsplit_span<F, NT, KR>();
  const int64_t items = static_cast<int64_t>(a.batch) * a.heads;
  const int sms = num_sms < kMaxRuns / 2 ? num_sms : kMaxRuns / 2;
  const int grid = a.split || items > 2 * sms ? sms : static_cast<int>((items + 1) / 2);
  auto kern = attn_decode_kernel<D, BS, F, NT, KR>;
  cudaError_t e =
      cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
  if (e != cudaSuccess) return e;
  e = launch_kernel(kern, dim3(grid), dim3(S::W * 32), kSmem, s, programmatic_after_kernel(s), a);
  if (e != cudaSuccess || !a.split) return e;
  return launch_kernel(attn_join_kernel<D, F, NT, S::TILE>, dim3(2 * grid), dim3(kJoinThreads), 0, s, true,
                       a);
}

template <int D, int BS, int F>
cudaError_t launch_f(AttnArgs& a, int rows, int64_t span, int num_sms, cudaStream_t s) {
  if constexpr (F == BNB4_F16)
    if (a.qtype == kQtNF4)
      return rows <= 8 ? launch_t<D, BS, F, 1, true>(a, span, num_sms, s)
                       : launch_t<D, BS, F, 2, true>(a, span, num_sms, s);
  return rows <= 8 ? launch_t<D, BS, F, 1, false>(a, span, num_sms, s)
                   : launch_t<D, BS, F, 2, false>(a, span, num_sms, s);
}

}  // namespace

// At most this many rows per (sequence, key/value head) run here, as many as the
// registers hold sums for; more go to the tensor-core kernel, whose tiles have
// 256 rows, padded or not.  At 16 rows and 12 sequences
// of about 3000 tokens this kernel takes 56 us, that one 73 (bf16) to 121 (fp16);
// with little cache to read the two are alike.
constexpr int64_t kMaxRows = 16;
// The workspace query knows no device: it splits for this many SMs, and so
// does the launch.
constexpr int kSms = 148;

static AttnArgs args_of(const bnb4_attn& p, int64_t* rows, int64_t* span) {
  const bnb4_kv_cache& c = *p.cache;
  AttnArgs a = {};
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
  a.causal = p.causal, a.qtype = c.qtype;
  a.window = p.window < (1 << 30) ? p.window : 1 << 30;
  a.page = make_div(static_cast<uint32_t>(c.page_size));
  a.scale_log2 = p.scale * 1.44269504088896f;
  a.ws = static_cast<float*>(p.workspace);
  *rows = static_cast<int64_t>(a.max_q) * a.group;
  // tokens that a row tile sees at most (a wide one: its queries' too)
  const int64_t own = *rows <= kMaxRows ? a.max_q : 256 / a.group + 2;
  *span = a.window > 0 && a.window + own + 15 < p.max_seq_len ? a.window + own + 15 : p.max_seq_len;
  return a;
}

size_t attn_workspace_bytes(const bnb4_attn& p) {
  int64_t rows, span;
  const AttnArgs a = args_of(p, &rows, &span);
  if (rows > kMaxRows) return attn_prefill_workspace(a, p.cache->head_dim, rows, span, kSms);
  const size_t rt = rows <= 8 ? 8 : 16;
  const bool kr = p.cache->dtype == BNB4_F16 && p.cache->qtype == BNB4_NF4;
  const int64_t whole = rows <= 8 ? (kr ? unsplit_span<BNB4_F16, 1, true>() : unsplit_span<BNB4_BF16, 1, false>())
                                  : (kr ? unsplit_span<BNB4_F16, 2, true>() : unsplit_span<BNB4_BF16, 2, false>());
  if (span <= whole) return 0;
  return sizeof(float) * 2 * kMaxRuns * rt * (static_cast<size_t>(p.cache->head_dim) + 2);
}

cudaError_t launch_attn(const bnb4_attn& p, int num_sms, int* err, cudaStream_t s,
                        uint64_t wait_limit_ns, int withhold) {
  const bnb4_kv_cache& c = *p.cache;
  int64_t rows, span;
  AttnArgs a = args_of(p, &rows, &span);
  a.err = err;
  a.wait_limit_ns = wait_limit_ns ? wait_limit_ns : kWaitLimitNs;
  a.withhold = withhold;
  if (rows > kMaxRows) return launch_attn_prefill(a, c, rows, span, kSms, s);
  const int rt = rows <= 8 ? 8 : 16;
#define BNB4_ATTN(DV, BSV)                                                               \
  return c.dtype == BNB4_F16 ? launch_f<DV, BSV, BNB4_F16>(a, rt, span, num_sms, s)      \
                             : launch_f<DV, BSV, BNB4_BF16>(a, rt, span, num_sms, s);
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
