// MLA decode over a cache held in e4m3 with one fp32 scale for each block of
// tokens, sm_103a.
//
// Mathematics.  With k8_t a cached token's 576 codes and c_t its scale,
//   s_t  = softmax_scale c_t <q, k8_t>
//   out  = sum_t p_t c_t k8_t[0:512] / sum_t p_t,   p_t = exp(s_t - max)
// so the scales never touch the codes: c_t multiplies the score's column and
// the probability.  Both products therefore run on the 8-bit tensor cores
// straight from the page as it lies in shared memory; nothing is converted.
// What they are multiplied with is split so that it loses nothing that matters:
//  * q (bf16, 8 significant bits) = hi + lo, two e4m3 numbers of 4 bits each,
//    after a power of two per row that puts the row's largest magnitude into
//    [128, 256).  The sum is exact for every element above 2^-9 of the row's
//    largest, and off by at most 2^-17 of the largest below.
//  * w_t = p_t c_t, scaled by a power of two for each row and block of 32
//    tokens that puts the block's largest into (2^7, 2^8], = hi + lo, both
//    e4m3: off by at most 2^-8 of w_t, as a bf16 probability, or 2^-17 of the
//    block's largest where that is more.  The block's exponent goes to the MMA
//    as its scale factor (block-scaled MMA), taken against a whole-numbered
//    reference of the row, in log2 units of p c.  It has 8 bits, so the
//    reference is set at an entry's first page and moves only when a later
//    score passes it by 2^40: O and the sums are hardly ever rescaled.  Both
//    are held times 2^-44, so that the p of a token whose c is 2^-100 fits.
// The sums of p_t, the maxima, scores and O are fp32.
//
// Layout of the work.  One CTA, 64 query rows, whole pages:
//  * S: the stacked operand [Q_hi; Q_lo] is the M = 128 rows of one MMA (A
//    from TMEM, 144 columns, so that only the page comes through shared
//    memory), B the page (64 tokens, K-major).  Rows r and r + 8 of each 16
//    TMEM lanes hold the hi and lo half of one head, which the 16x256b load
//    hands to one thread in different registers.  With 16 or 32 rows the heads
//    are repeated over the lanes; the warps that share a row take slices of
//    the page's tokens.
//  * O^T = V^T W^T: M = 128 dims (four blocks), the page itself as M-major A.
//    Up to 32 rows B is [rows hi; rows lo] x 64 tokens and O^T has a column
//    for each half, so that V is read once; with 64 rows that would need all
//    of TMEM, B is rows x [64 hi | 64 lo] and both halves add into 4 x 64
//    columns, a block of V being kept in the tensor core's collector between
//    them.
// Rows above 64 are cut into tiles; the CTAs of the tiles take the same page
// ranges at the same time, so that a page read by one is in L2 for the others.
//
// Warp roles: warps 0-7 softmax and epilogue (two for each TMEM lane quarter,
// with half a page's tokens each, or less), all on the same page, warp 8 the
// TMA producer, warp 9 the score MMA issuer and TMEM owner, warp 10 the P.V
// MMA issuer, warp 11 the scales (a ring beside the page stages).  Two groups
// of four warps on alternate pages, 16 warps and pages overlapped within a
// warp were slower (by 5 to 13 %: warps at the same place share the fetch of
// the code).  Every wait is bounded (globaltimer): on expiry the kernel records
// MLA_ERR_DEVICE_TIMEOUT, lets in-flight copies land, frees TMEM and returns.
//
// What bounds it, per CTA and page of 64 tokens with 64 rows: the MMAs take
// 576 (S) + 608 cycles, the shared memory 1100 to feed them (144 KB a page),
// the softmax warps about 1700: reading S to its maxima 650, barrier 120 to
// 190, weights 600, fences and waits 270; the next page's S is there before
// they ask for it.  132 x 2 x 128 heads over 8192 tokens take 430 to 467 us
// without their plan, as the card's power limit lets: 1.3 to 1.4 PFLOP/s of 2 x
// 1088 a row and key, and the split doubles what the MMAs do.
// Tried and not kept there (us for that call; the kernel at the time in
// brackets): two score tiles, with the query's last 128 dims in shared memory
// for them, 456 (435); block exponents guessed from the pages before and the
// maxima checked after the weights 463 (440, a guess of 128 fails too often);
// all of a query's loads at once 513 (477).  With up to 32 rows the cache's
// bytes bound it: over 65536 tokens 8 x 16 heads take 53 us (5.7 TB/s), 8 x 32
// heads 57 (5.4 TB/s), without plan and combine.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include <mutex>
#include <type_traits>

#include "mla.h"
#include "mla_fp8.h"
#include "ptx_sm103.cuh"

namespace mla {
namespace {

constexpr int kFThreads = 384;
constexpr int kFSoftWarps = 8;    // two for each TMEM lane quarter
constexpr int kFSoftThreads = 32 * kFSoftWarps;
constexpr int kFProducerWarp = 8;
constexpr int kFMmaWarp = 9;      // score MMAs; owns TMEM
constexpr int kFPvWarp = 10;      // P.V MMAs
constexpr int kFScaleWarp = 11;
constexpr uint64_t kFWaitNs = 2000000000ull;  // 2 s per wait
constexpr uint64_t kFDrainNs = 2000000ull;    // settle time after an abort
constexpr float kFLn2 = 0.69314718055994530942f;
constexpr float kTarget = 8.0f;   // log2 that the largest weight of a block of 32 tokens may have
constexpr float kSlack = 40.0f;   // growth of the maximum over the reference that needs no rescale
constexpr int kBlockMin = -82;    // smallest block exponent relative to the reference
// Scales whose logarithm is taken: 2^-100 (the least that the append stores) to
// 2^60.  p = w / c is then up to 2^100 times w, and w up to 2^(8 + 40) over the
// reference: O and the sums of p are both held times 2^-44 (O by V's scale factor
// in the MMA), which keeps 2^20 such p, and one p at c = 2^60, finite and normal.
constexpr float kLogMin = 7.8886090522101181e-31f, kLogMax = 1.152921504606847e18f;
constexpr int kSumShift = 44;
constexpr float kTotShift = 17592186044416.0f;   // 2^44
static_assert(kBlockMin + 127 - kSumShift >= 1, "the sums' factor of a block stays normal");

constexpr int kFStages = 5;
constexpr uint32_t kFBox = 64 * 128;                       // 64 tokens x 128 dims, 128-byte swizzle
constexpr uint32_t kFRope = 4 * kFBox;                     // 64 tokens x 64 dims, 64-byte swizzle
constexpr uint32_t kFStageBytes = kFRope + 64 * 64;        // one page: 36,864
constexpr uint32_t kFTmemCols = 512;
constexpr uint32_t kFColQ = 0;                             // [0, 144): Q, four codes a column
constexpr uint32_t kFColSfa = 144;                         // scales of V (2^-44)
constexpr uint32_t kFColSfb = 148;                         // 2 x 4 columns: scales of W
constexpr uint32_t kFColS = 192;                           // one or two score tiles of 64 columns

template <int kR>
struct FShape {
  static_assert(kR == 16 || kR == 32 || kR == 64, "16, 32 or 64 query rows");
  static constexpr int kSlices = 128 / kR;                   // warps that share a row
  static constexpr int kTok = kR / 2;                        // tokens of a page a warp takes
  // up to 32 rows the hi and lo weights are separate rows of W^T and separate
  // columns of O^T (one pass over V); 64 rows have no TMEM for that
  static constexpr bool kWide = kR <= 32;
  static constexpr uint32_t kCols = kWide ? 2 * kR : kR;     // O^T columns of a 128-dim block
  static constexpr uint32_t kColO = 512 - 4 * kCols;
  static constexpr uint32_t kSBufs = kR == 16 ? 2 : 1;       // score tiles that fit
  static constexpr uint32_t kWBytes = (uint32_t)kR * 128u;   // W^T of a page
  static constexpr uint32_t kW = kFStages * kFStageBytes;    // 2 W^T tiles
  static constexpr uint32_t kSfb = kW + 2 * kWBytes;         // 2 x 512: block exponents of W
  // with 16 rows the four lane quarters hold the same query: split once, handed
  // round in shared memory (2 halves x 18 steps x 32 lanes x 16 bytes)
  static constexpr bool kShareQ = kR == 16;
  static constexpr uint32_t kQSplit = kSfb + 1024;
  static constexpr uint32_t kScale = kQSplit + (kShareQ ? 18432 : 0);   // ring of 64 x {c, log2 c}
  static constexpr uint32_t kTop = kScale + kFStages * 512;  // 3 x u32[R] maxima that pass
  static constexpr uint32_t kBlk = kTop + 768;               // 2 x float[kSlices][R] maxima
  static constexpr uint32_t kSum = kBlk + 1024;              // float[kSlices][R] sums
  static constexpr uint32_t kFac = kSum + 512;               // float[R] factors of O^T's columns
  static constexpr uint32_t kQfac = kFac + 256;              // float[R] factors of the scores
  static constexpr uint32_t kBar = kQfac + 256;
  static constexpr uint32_t kMisc = kBar + 8 * 24;           // TMEM slot, abort flag
  static constexpr uint32_t kSmemAlloc = kMisc + 16 + 1024;
  static_assert(kFColS + 64 * kSBufs <= kColO, "TMEM columns");
  static_assert(kW % 1024 == 0 && kWBytes % 1024 == 0, "swizzled buffers need 1 KB alignment");
  static_assert(kSmemAlloc <= 232448, "shared memory");
};

enum FBar : uint32_t {
  F_FULL = 0,                 // [5] page loaded (TMA tx) and its scales written (scale warp)
  F_EMPTY = kFStages,         // [5] page consumed (MMA commit after its P.V)
  F_SFULL = 2 * kFStages,     // [2] score tile ready (MMA commit); scales and the W^T buffer
                              // seen (score warp)
  F_SEMPTY = F_SFULL + 2,     // [2] score tile read (softmax warps)
  F_PFULL = F_SEMPTY + 2,     // [2] W^T written, O^T rescaled (softmax warps)
  F_PEMPTY = F_PFULL + 2,     // [2] the P.V of the tile's page done (MMA commit)
  F_QFULL = F_PEMPTY + 2,     // Q of the entry in TMEM (softmax warps)
  F_QEMPTY,                   // the entry's last score MMA done (MMA commit)
  F_TEARDOWN,
  F_COUNT,
};
static_assert(F_COUNT <= 24, "barrier space");

struct FCtx {
  uint32_t sbase, tmem, abort_addr, bar0;
  int* err;
  __device__ __forceinline__ uint32_t bar(uint32_t i) const { return bar0 + 8u * i; }
};

// The part of a wait that is seldom reached, out of line: the page loop's code
// is fetched by twelve warps in four roles, and its length shows (with this,
// f_rescale and f_zero_rows inline, 87 KB instead of 82 in all, 132 x 2 x 128
// heads over 8192 tokens take 477 us instead of 453).
__device__ __noinline__ bool f_wait_long(uint32_t bar, uint32_t parity, uint32_t abort_addr,
                                         int* err) {
  const uint64_t t0 = ptx::globaltimer();
  for (uint32_t i = 0;; ++i) {
    if ((i & 63u) == 0u) {
      if (ptx::ld_shared_u32_volatile(abort_addr) != 0u) return false;
      if (ptx::globaltimer() - t0 > kFWaitNs) {
        atomicCAS(err, 0, MLA_ERR_DEVICE_TIMEOUT);
        ptx::st_shared_u32(abort_addr, 1u);
        return false;
      }
    }
    if (ptx::mbar_try_wait(bar, parity)) return true;
  }
}
__device__ __forceinline__ bool f_wait(const FCtx& x, uint32_t bar, uint32_t parity) {
  if (ptx::mbar_try_wait(bar, parity)) return true;
  return f_wait_long(bar, parity, x.abort_addr, x.err);
}
__device__ __forceinline__ bool f_wait_warp(const FCtx& x, uint32_t bar, uint32_t parity) {
  const bool ok = f_wait(x, bar, parity);
  return __all_sync(0xffffffffu, ok);
}
// The softmax warps meet on a hardware barrier.  They all run the same number
// of pages and entries and never leave early: a wait that gave up (or finds
// the abort flag) lets its warp go on with stale values, so every warp arrives
// at every barrier and the kernel ends with the error recorded.
__device__ __forceinline__ void f_sync() {
  __syncwarp();
  ptx::named_sync(1, kFSoftThreads);
}
__device__ __forceinline__ bool f_sync_or(bool v) {
  __syncwarp();
  return ptx::named_sync_or(1, kFSoftThreads, v);
}

// The combine's look at the plan's header: a word a lane, one request a warp
// (with one a word the line that the whole grid reads becomes a hot spot: one
// entry of 4096 tokens with 128 heads 16.8 -> 21.5 us), and whether the plan is
// one for this call.
__device__ __forceinline__ int f_plan_head(const int32_t* plan, int lane) {
  return __ldcg(plan + (lane & (H_WORDS - 1)));
}
__device__ __forceinline__ bool f_plan_ours(int head, const Fp8Params& prm, int lane) {
  const int tiles = f8_tiles(prm.s_q, prm.h_q);
  int want = head;
  if (lane == H_MAGIC) want = kF8PlanMagic;
  if (lane == H_BATCH) want = prm.batch;
  if (lane == H_SQ) want = prm.s_q;
  if (lane == H_HQ) want = prm.h_q;
  if (lane == H_TILES) want = tiles;
  if (lane == H_GT) want = prm.workers / tiles;
  if (lane == H_NCLUSTERS) want = prm.workers;
  return __all_sync(0xffffffffu, head == want);
}

struct FWork {
  int b0, p0, b1, p1, split0, tile;
  const int32_t* items;
  int64_t stotal;
};

// This CTA's pages in order; g counts them.
struct FPages {
  SegIter it;
  uint32_t g;
  int b, pg, pb, pe;
  bool valid;
  __device__ __forceinline__ void init(const FWork& w) {
    it = SegIter{w.b0, w.p0, w.b1, w.p1, w.items};
    g = 0;
    valid = it.next(b, pb, pe);
    pg = pb;
  }
  __device__ __forceinline__ void advance() {
    ++g;
    if (++pg == pe) {
      valid = it.next(b, pb, pe);
      pg = pb;
    }
  }
};

// Pool page of page pg of entry b.  Entries past max_pages are never read:
// such a page (and one outside the pool) is reported and served from page 0.
__device__ __forceinline__ int f_page_of(const FCtx& x, const Fp8Params& prm, int b, int pg,
                                         bool report) {
  const int page = pg < prm.max_pages ? prm.block_table[(size_t)b * prm.max_pages + pg] : -1;
  if ((unsigned)page < (unsigned)prm.num_pages) return page;
  if (report) atomicCAS(x.err, 0, MLA_ERR_DEVICE_BOUNDS);
  return 0;
}

// ------------------------------------------------------------------ producer
// hint: with one tile a page is read once, so it leaves L2 first.
__device__ __forceinline__ void f_producer(const FCtx& x, const FWork& w, const Fp8Params& prm,
                                           const CUtensorMap* lat, const CUtensorMap* rope,
                                           bool once) {
  const uint64_t policy = ptx::policy_evict_first();
  FPages cur;
  cur.init(w);
  while (cur.valid) {
    const int page = f_page_of(x, prm, cur.b, cur.pg, true);
    const uint32_t g = cur.g, s = g % kFStages;
    if (!f_wait(x, x.bar(F_EMPTY + s), ((g / kFStages) & 1u) ^ 1u)) return;
    const uint32_t bar = x.bar(F_FULL + s), st = x.sbase + s * kFStageBytes;
    ptx::mbar_arrive_expect_tx(bar, kFStageBytes);
    const int row = page * kPageTokens;
#pragma unroll 1
    for (uint32_t j = 0; j < 4; ++j) {
      if (once)
        ptx::tma_load_2d_hint(st + j * kFBox, lat, 128 * (int)j, row, bar, policy);
      else
        ptx::tma_load_2d(st + j * kFBox, lat, 128 * (int)j, row, bar);
    }
    if (once)
      ptx::tma_load_2d_hint(st + kFRope, rope, kDv, row, bar, policy);
    else
      ptx::tma_load_2d(st + kFRope, rope, kDv, row, bar);
    cur.advance();
  }
}

// The scales of a page's tokens, two a lane, with their logarithms (which only
// choose the running maximum; its error cancels).  Tokens past the length get
// zero.  Four pages' loads are in flight together.
template <int kR>
__device__ __forceinline__ void f_scales(const FCtx& x, const FWork& w, const Fp8Params& prm,
                                         int lane) {
  constexpr int kBatch = 4;
  FPages cur;
  cur.init(w);
  const int per_page = kPageTokens >> prm.scale_shift;
  while (cur.valid) {
    int page[kBatch], left[kBatch], n = 0;
    const uint32_t g0 = cur.g;
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      page[k] = left[k] = 0;
      if (cur.valid) {
        page[k] = f_page_of(x, prm, cur.b, cur.pg, false);
        left[k] = prm.seqlens[cur.b] - cur.pg * kPageTokens;
        n = k + 1;
        cur.advance();
      }
    }
    float c0[kBatch], c1[kBatch];
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      const float* src = prm.scales + (int64_t)page[k] * per_page;
      c0[k] = 2 * lane < left[k] ? src[(2 * lane) >> prm.scale_shift] : 0.f;
      c1[k] = 2 * lane + 1 < left[k] ? src[(2 * lane + 1) >> prm.scale_shift] : 0.f;
    }
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      if (k >= n) break;
      const uint32_t g = g0 + k, s = g % kFStages;
      if (!f_wait_warp(x, x.bar(F_EMPTY + s), ((g / kFStages) & 1u) ^ 1u)) return;
      const float l0 = __log2f(fminf(fmaxf(fabsf(c0[k]), kLogMin), kLogMax));
      const float l1 = __log2f(fminf(fmaxf(fabsf(c1[k]), kLogMin), kLogMax));
      ptx::st_shared_v4(x.sbase + FShape<kR>::kScale + s * 512u + (uint32_t)lane * 16u,
                        __float_as_uint(c0[k]), __float_as_uint(l0), __float_as_uint(c1[k]),
                        __float_as_uint(l1));
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(x.bar(F_FULL + s));
    }
  }
}

// ------------------------------------------------------------------ MMA issuers
// S(g) = [Q_hi; Q_lo] K^T once page g is loaded, its score tile is free and
// the entry's Q is there.
template <int kR>
__device__ __forceinline__ void f_mma_s(const FCtx& x, const FWork& w, int lane) {
  using S = FShape<kR>;
  constexpr uint32_t id_s = ptx::idesc_f8(128, 64, 0, 0, 0, 0);
  FPages sc;
  sc.init(w);
  uint32_t sq = 0;   // entries whose score MMAs are all issued (Q uses)
  while (sc.valid) {
    const uint32_t g = sc.g, s = g % kFStages;
    if (sc.pg == sc.pb && !f_wait_warp(x, x.bar(F_QFULL), sq & 1u)) return;
    if (!f_wait_warp(x, x.bar(F_FULL + s), (g / kFStages) & 1u)) return;
    const uint32_t sb = g % S::kSBufs, su = g / S::kSBufs;
    if (su >= 1 && !f_wait_warp(x, x.bar(F_SEMPTY + sb), (su & 1u) ^ 1u)) return;
    ptx::tc_fence_after();
    const uint32_t st = x.sbase + s * kFStageBytes;
    const uint32_t d_s = x.tmem + kFColS + sb * 64u;
    const uint64_t k_desc = ptx::smem_desc(st, 16, 1024, ptx::kLayoutSw128);
#pragma unroll
    for (uint32_t box = 0; box < 4; ++box)   // 32 dims a step
      ptx::mma8_ts4_elect(d_s, x.tmem + kFColQ + 32u * box, k_desc + box * (kFBox >> 4), id_s, box);
    ptx::mma8_ts2_elect(d_s, x.tmem + kFColQ + 128u,
                        ptx::smem_desc(st + kFRope, 16, 512, ptx::kLayoutSw64), id_s, 1u);
    ptx::mma_commit_elect(x.bar(F_SFULL + sb));
    // Hands on what this warp has seen: the page's scales (F_FULL), and that
    // the page's W^T buffer is free, the P.V of page g - 2 being done.
    if (g >= 2 && !f_wait_warp(x, x.bar(F_PEMPTY + (g & 1u)), ((g >> 1) & 1u) ^ 1u)) return;
    __syncwarp();
    if (lane == 0) ptx::mbar_arrive(x.bar(F_SFULL + sb));
    if (sc.pg == sc.pe - 1) {
      ptx::mma_commit_elect(x.bar(F_QEMPTY));
      ++sq;
    }
    sc.advance();
  }
}

// O^T += V^T W^T once page g's weights are written; the commits hand the stage
// back to the producer and the W^T buffer to the softmax warps.
template <int kR>
__device__ __forceinline__ void f_mma_o(const FCtx& x, const FWork& w) {
  using S = FShape<kR>;
  FPages oc;
  oc.init(w);
  while (oc.valid) {
    const uint32_t g = oc.g, s = g % kFStages;
    if (!f_wait_warp(x, x.bar(F_PFULL + (g & 1u)), (g >> 1) & 1u)) return;
    ptx::tc_fence_after();
    const bool first = (oc.pg == oc.pb);
    const uint32_t st = x.sbase + s * kFStageBytes;
    const uint32_t wt = x.sbase + S::kW + (g & 1u) * S::kWBytes;
    const uint32_t sfa = x.tmem + kFColSfa, sfb = x.tmem + kFColSfb + 4u * (g & 1u);
    ptx::tmem_cp_32x128b_x4_elect(
        sfb, ptx::smem_desc(x.sbase + S::kSfb + (g & 1u) * 512u, 16, 128, ptx::kLayoutNone));
    // V^T block mb: dims [128 mb, +128) = one box, two steps of 32 tokens (four
    // 8-token groups 1 KB apart).  W^T rows: 64 tokens of the hi or of the lo
    // half, or 64 hi then 64 lo tokens.
    const uint64_t v_desc = ptx::smem_desc(st, kFBox, 1024, ptx::kLayoutSw128);
    const uint64_t w_desc = S::kWide ? ptx::smem_desc(wt, 16, 512, ptx::kLayoutSw64)
                                     : ptx::smem_desc(wt, 16, 1024, ptx::kLayoutSw128);
    constexpr uint32_t id_o = ptx::idesc_mx8(128, (int)S::kCols, 1, 0, 0);
#pragma unroll
    for (uint32_t mb = 0; mb < 4; ++mb) {
      const uint32_t d = x.tmem + S::kColO + S::kCols * mb, add = first ? 0u : 1u;
      if constexpr (S::kWide)
        ptx::mma8_scaled_x2_elect(d, v_desc + mb * (kFBox >> 4), w_desc, id_o, sfa, sfb, add);
      else
        ptx::mma8_scaled_x4_elect(d, v_desc + mb * (kFBox >> 4), w_desc, id_o, sfa, sfb, add);
    }
    ptx::mma_commit_elect(x.bar(F_EMPTY + s));
    ptx::mma_commit_elect(x.bar(F_PEMPTY + (g & 1u)));
    oc.advance();
  }
}

// ------------------------------------------------------------------ softmax
// hi + lo of two values as packed e4m3 pairs: hi the nearest, lo the rest.
__device__ __forceinline__ void f_split(float a, float b, uint32_t& hi, uint32_t& lo) {
  const __half2 h = __floats2half2_rn(a, b);
  const __nv_fp8x2_storage_t h8 =
      __nv_cvt_halfraw2_to_fp8x2(static_cast<__half2_raw>(h), __NV_SATFINITE, __NV_E4M3);
  const __half2 rest = __hsub2(h, __half2(__nv_cvt_fp8x2_to_halfraw2(h8, __NV_E4M3)));
  hi = h8;
  lo = __nv_cvt_halfraw2_to_fp8x2(static_cast<__half2_raw>(rest), __NV_SATFINITE, __NV_E4M3);
}

// Out of line as well.  Columns of this warp's two blocks of O^T times their rows' factors (of
// row l % R in lane l of a0, of row l + 32 in a1):
template <int kR>
__device__ __noinline__ void f_rescale(uint32_t o_base, float a0, float a1) {
#pragma unroll 1
  for (int ch = 0; ch < (int)(2 * FShape<kR>::kCols / 32); ++ch) {
    const float av = (kR == 64 && (ch & 1)) ? a1 : a0;
    uint32_t o[32];
    ptx::tmem_ld32_wait(o_base + 32u * (uint32_t)ch, o);
#pragma unroll
    for (int j = 0; j < 32; ++j)
      o[j] = __float_as_uint(__uint_as_float(o[j]) * __shfl_sync(0xffffffffu, av, j % kR));
    ptx::tmem_st32(o_base + 32u * (uint32_t)ch, o);
  }
  ptx::tmem_wait_st();
}
// The value rows from token tz on of the page at st.
__device__ __noinline__ void f_zero_rows(uint32_t st, int tz, int tid) {
  const int n16 = (kPageTokens - tz) * 4 * 8;   // rows x 4 boxes x 8 pieces of 16 bytes
  for (int idx = tid; idx < n16; idx += kFSoftThreads)
    ptx::st_shared_v4(st + (uint32_t)((idx >> 3) & 3) * kFBox + (uint32_t)(tz + (idx >> 5)) * 128u +
                          (uint32_t)(idx & 7) * 16u,
                      0u, 0u, 0u, 0u);
}

template <int kR>
__device__ __forceinline__ void f_softmax(const FCtx& x, const FWork& w, const Fp8Params& prm,
                                          int warp, int lane) {
  using S = FShape<kR>;
  constexpr int kJ = S::kTok / 8;                         // groups of 8 tokens in a warp's slice
  constexpr int kHeadWarps = kR / 16;
  const int quarter = warp & 3, grp = warp >> 2;
  const int tl = 32 * quarter + lane;                     // TMEM lane
  const int tid = 32 * warp + lane;
  const uint32_t lanes = (uint32_t)(32 * quarter) << 16;
  const int hb = 16 * (quarter % kHeadWarps);             // first row of this warp
  const int slice = grp * (4 / kHeadWarps) + quarter / kHeadWarps;
  const int tok0 = slice * S::kTok;                       // its tokens of a page: [tok0, +kTok)
  const int r8 = lane >> 2, cq = lane & 3;                // fragment row and column pair
  const int rows = prm.s_q * prm.h_q - w.tile * kF8TileRows;   // rows of this tile (may exceed R)
  const int n_rows = rows < kR ? rows : kR;

  SegIter it{w.b0, w.p0, w.b1, w.p1, w.items};
  int b, pb, pe;
  uint32_t g = 0, nq = 0, n_item = 0;
  // where this thread's weights go: rows hb + r8 (and 8 further), tokens 2 cq,
  // 2 cq + 1 of each 8; the 16-byte chunk is swizzled by the row
  const uint32_t w_base =
      x.sbase + S::kW + 2u * (uint32_t)cq + (uint32_t)(tok0 & 8) +
      (S::kWide ? (uint32_t)(hb + r8) * 64u + (((uint32_t)(r8 >> 1) & 3u) << 4)
                : (uint32_t)(hb + r8) * 128u + ((uint32_t)r8 << 4));
  const uint32_t w_at[2] = {w_base ^ (uint32_t)(tok0 & ~15),
                            w_base ^ (uint32_t)((tok0 & ~15) + 16)};
  // The entry's Q into TMEM once the previous entry's last score MMA is done:
  // as fragments, so that four threads read 64 consecutive bytes of a row and
  // the hi and lo codes of a thread's 8 dims are its own four registers.  Of
  // the 16 rows of a lane quarter each of its two warps takes 8.  With more than
  // 16 rows a row is read twice (the second time mostly from L2): its largest
  // magnitude first.  The rows' softmax_scale log2(e) / 2^k go to a table that a
  // later barrier publishes.
  auto load_q = [&](int qb) {
    const int row = hb + 8 * grp + r8;
    const uint4* src = reinterpret_cast<const uint4*>(
        static_cast<const __nv_bfloat16*>(prm.q) +
        ((int64_t)qb * prm.s_q * prm.h_q + w.tile * kF8TileRows + (row < n_rows ? row : 0)) * kDqk +
        8 * cq);
    // Up to 16 rows the four lane quarters hold the same rows: each reads, and
    // later splits, every fourth step, all at once, and the maxima meet in shared
    // memory.  Else the loops are kept short, for the instruction cache.
    constexpr int kMine = 5;
    uint4 mine[S::kShareQ ? kMine : 1];
    uint32_t top2 = 0;   // magnitudes of bf16 pairs order as unsigned numbers (NaN above all)
    auto widen = [&](const uint4& raw) {
      const uint32_t u[4] = {raw.x, raw.y, raw.z, raw.w};
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const uint32_t v2 = u[c] & 0x7fff7fffu;
        top2 = __vmaxu2(top2, v2);
      }
    };
    if constexpr (S::kShareQ) {
#pragma unroll
      for (int k = 0; k < kMine; ++k)
        mine[k] = quarter + 4 * k < 18 ? src[4 * (quarter + 4 * k)] : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
      for (int k = 0; k < kMine; ++k) widen(mine[k]);
    } else {
#pragma unroll 1
      for (int k0 = 0; k0 < 18; k0 += 9) {
        uint4 raw[9];
#pragma unroll
        for (int k = 0; k < 9; ++k) raw[k] = src[4 * (k0 + k)];
#pragma unroll
        for (int k = 0; k < 9; ++k) widen(raw[k]);
      }
    }
    float big = __uint_as_float(max(top2 << 16, top2 & 0xffff0000u));
    big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, 1));
    big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, 2));
    if constexpr (S::kShareQ) {
      // (the table of sums is free: its last readers are behind a barrier, and
      // the one before the codes are read comes before its next writers)
      const uint32_t at = x.sbase + S::kSum + (uint32_t)row * 4u;
      if (cq == 0) ptx::st_shared_u32(at + (uint32_t)quarter * 64u, __float_as_uint(big));
      f_sync();
#pragma unroll
      for (uint32_t k = 0; k < 4; ++k)
        big = fmaxf(big, __uint_as_float(ptx::ld_shared_u32_volatile(at + k * 64u)));
    }
    // 2^(7 - floor(log2 big)) by its exponent field, and the inverse; a row that
    // holds an infinity becomes NaN (the conversions would saturate it)
    uint32_t e = (__float_as_uint(big) >> 23) & 255u;
    const float mul = row >= n_rows ? 0.f
                      : e == 255u   ? NAN
                                    : __uint_as_float((261u - max(e, 10u)) << 23);
    e = min(max(e, 10u), 254u);
    if (quarter < kHeadWarps && cq == 0)
      ptx::st_shared_u32(x.sbase + S::kQfac + (uint32_t)row * 4u,
                         __float_as_uint(prm.scale_log2 * __uint_as_float((e - 7u) << 23)));
    // 8 dims of step k as codes: hi and lo of dims 0-3, 4-7
    auto split8 = [&](const uint4& raw) {
      const uint32_t u[4] = {raw.x, raw.y, raw.z, raw.w};
      uint32_t hi[4], lo[4];
#pragma unroll
      for (int c = 0; c < 4; ++c)
        f_split(__uint_as_float(u[c] << 16) * mul,
                       __uint_as_float(u[c] & 0xffff0000u) * mul, hi[c], lo[c]);
      return make_uint4(hi[0] | (hi[1] << 16), hi[2] | (hi[3] << 16), lo[0] | (lo[1] << 16),
                        lo[2] | (lo[3] << 16));
    };
    const uint32_t dst = x.tmem + lanes + ((uint32_t)(16 * grp) << 16) + kFColQ;
    if constexpr (S::kShareQ) {
      const uint32_t share = x.sbase + S::kQSplit + (uint32_t)(grp * 18 * 512 + lane * 16);
#pragma unroll
      for (int k = 0; k < kMine; ++k) {
        const uint4 c = split8(mine[k]);
        if (quarter + 4 * k < 18)
          ptx::st_shared_v4(share + (uint32_t)(quarter + 4 * k) * 512u, c.x, c.y, c.z, c.w);
      }
      f_wait(x, x.bar(F_QEMPTY), (nq & 1u) ^ 1u);
      f_sync();
#pragma unroll
      for (int k = 0; k < 18; ++k) {
        const uint4 c = ptx::ld_shared_v4u(share + (uint32_t)k * 512u);
        ptx::tmem_st16x256b(dst + 8u * (uint32_t)k, c.x, c.y, c.z, c.w);
      }
    } else {
      uint4 raw[3], next[3];                                // three steps on the way
#pragma unroll
      for (int k = 0; k < 3; ++k) next[k] = src[4 * k];
      f_wait(x, x.bar(F_QEMPTY), (nq & 1u) ^ 1u);
      __syncwarp();
#pragma unroll 1
      for (int k0 = 0; k0 < 18; k0 += 3) {
        const int k1 = k0 < 15 ? k0 + 3 : 15;
#pragma unroll
        for (int k = 0; k < 3; ++k) {
          raw[k] = next[k];
          next[k] = src[4 * (k1 + k)];
        }
#pragma unroll
        for (int k = 0; k < 3; ++k) {
          const uint4 c = split8(raw[k]);
          ptx::tmem_st16x256b(dst + 8u * (uint32_t)(k0 + k), c.x, c.y, c.z, c.w);
        }
      }
    }
    ptx::tmem_wait_st();
    ptx::tc_fence_before();
    __syncwarp();
    if (lane == 0) ptx::mbar_arrive(x.bar(F_QFULL));
    ++nq;
  };

  // V's scales
  if (grp == 0) {
#pragma unroll
    for (uint32_t k = 0; k < 4; ++k)
      ptx::tmem_st1(x.tmem + lanes + kFColSfa + k, 0x01010101u * (uint32_t)(127 - kSumShift));
    ptx::tmem_wait_st();
    ptx::tc_fence_before();
  }
  uint32_t stg = 0, top_i = 0;                            // page stage; g % 3
  if (tid < kR) {
#pragma unroll
    for (int k = 0; k < 3; ++k)
      ptx::st_shared_u32(x.sbase + S::kTop + (uint32_t)(k * kR + tid) * 4u, 0u);
  }
  bool have = it.next(b, pb, pe);
  if (have) load_q(b);
  f_sync();
  while (have) {
    // of this thread's two fragment rows
    float fac[2], m[2];
    uint64_t sum[2];                                        // over even and odd tokens
    int nv[2];
    const int L = prm.seqlens[b];
    const int n_min = L - prm.s_q + 1;                      // keys the first query token sees
    const int P_total = w.items[b * kItemWords + 0];
    const int ns = w.items[b * kItemWords + 1], slot0 = w.items[b * kItemWords + 2];
    const bool direct = (ns == 1);
    const int64_t slot = (int64_t)w.tile * w.stotal + slot0 + (n_item == 0 ? w.split0 : 0);
    const bool slot_ok = direct || (slot >= 0 && slot < f8_slots(prm.workers));
    float* lse_at[2];                                       // of this thread's rows
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      // written before the barriers of the previous entry's end (or the one above)
      fac[h] = __uint_as_float(
          ptx::ld_shared_u32_volatile(x.sbase + S::kQfac + (uint32_t)(hb + 8 * h + r8) * 4u));
      const int row = w.tile * kF8TileRows + hb + 8 * h + r8, qi = row / prm.h_q;
      nv[h] = hb + 8 * h + r8 < n_rows ? n_min + qi : L;
      lse_at[h] = direct ? prm.lse + (((int64_t)b * prm.h_q + (row - qi * prm.h_q)) * prm.s_q + qi)
                         : prm.ws_lse + (slot * kR + hb + 8 * h + r8);
      m[h] = -INFINITY;                                     // the reference maximum
      sum[h] = 0;
    }
    const int pm = n_min > 0 ? n_min / kPageTokens : 0;     // pages before it are seen by all rows
    // every warp follows every row's reference: lane l that of row l % R and,
    // for R = 64, of row l + 32
    float mt[2] = {-INFINITY, -INFINITY};

    for (int pg = pb; pg < pe; ++pg, ++g) {
      const uint32_t wb = g & 1u;
      if (tid < kR)   // next page's table (its last readers have passed the last barrier)
        ptx::st_shared_u32(
            x.sbase + S::kTop + (uint32_t)((top_i == 2 ? 0u : top_i + 1u) * kR + tid) * 4u, 0u);
      const uint32_t sb = g % S::kSBufs;
      f_wait(x, x.bar(F_SFULL + sb), (g / S::kSBufs) & 1u);
      __syncwarp();
      ptx::tc_fence_after();
      uint64_t sc[kJ], v[2][kJ];                            // scales; q.k c over fac
      float z[2];                                           // the slice's maxima of s + log2 c
      {
        uint64_t ls[kJ];
        uint32_t r[8 * kJ];
        const uint32_t ring = x.sbase + S::kScale + stg * 512u + (uint32_t)(tok0 + 2 * cq) * 8u;
#pragma unroll
        for (int j = 0; j < kJ; ++j) {
          const uint4 u = ptx::ld_shared_v4u(ring + (uint32_t)j * 64u);
          sc[j] = (uint64_t)u.z << 32 | u.x;
          ls[j] = (uint64_t)u.w << 32 | u.y;
        }
        ptx::tmem_ld16x256b_pair_wait(x.tmem + lanes + kFColS + sb * 64u + (uint32_t)tok0, r);
        ptx::tc_fence_before();
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(x.bar(F_SEMPTY + sb));
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int j = 0; j < kJ; ++j) {
            const uint32_t* q = r + 4 * kJ * h + 4 * j;
            v[h][j] = ptx::f2_mul(
                ptx::f2_add((uint64_t)q[1] << 32 | q[0], (uint64_t)q[3] << 32 | q[2]), sc[j]);
          }
        if (pg >= pm) {                                     // keys some row does not see
#pragma unroll
          for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int j = 0; j < kJ; ++j) {
              const int key = pg * kPageTokens + tok0 + 8 * j + 2 * cq;
              float v0, v1;
              ptx::f2_unpack(v[h][j], v0, v1);
              v[h][j] = ptx::f2_pack(key < nv[h] ? v0 : -INFINITY, key + 1 < nv[h] ? v1 : -INFINITY);
            }
          // Past the end of the sequence the last page's slots hold stale codes,
          // NaN among them: their weights are 0, but 0 * NaN is NaN in the MMA,
          // so those value rows are zeroed (the score MMAs have read the page).
          if (pg == P_total - 1 && (L & (kPageTokens - 1)) != 0)
            f_zero_rows(x.sbase + stg * kFStageBytes, L & (kPageTokens - 1), tid);
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const uint64_t f2 = ptx::f2_pack(fac[h], fac[h]);
          z[h] = -INFINITY;
#pragma unroll
          for (int j = 0; j < kJ; ++j) {
            float z0, z1;
            ptx::f2_unpack(ptx::f2_fma(v[h][j], f2, ls[j]), z0, z1);
            z[h] = ptx::max3(z[h], z0, z1);
          }
          z[h] = fmaxf(z[h], __shfl_xor_sync(0xffffffffu, z[h], 1));
          z[h] = fmaxf(z[h], __shfl_xor_sync(0xffffffffu, z[h], 2));
        }
      }
      const uint32_t blk = x.sbase + S::kBlk + wb * 512u;
      if (kR < 64 && cq == 0) {                             // a block of 32 tokens is 2 or 4 warps'
#pragma unroll
        for (int h = 0; h < 2; ++h)
          ptx::st_shared_u32(blk + (uint32_t)(slice * kR + hb + 8 * h + r8) * 4u,
                             __float_as_uint(z[h]));
      }
      // The reference of a row moves only when it is passed by more than
      // kSlack (or at an entry's first page).  Who passes it puts its maximum
      // into the page's table, as an unsigned number of the same order, 0 for
      // none; the barrier tells everyone whether there is any.
      const uint32_t top = x.sbase + S::kTop + top_i * (uint32_t)(4 * kR);
      const bool pass = z[0] > m[0] + kSlack || z[1] > m[1] + kSlack;
      if (pass && cq == 0) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int s = __float_as_int(z[h]);
          if (z[h] > m[h] + kSlack)
            ptx::max_shared_u32(top + (uint32_t)(hb + 8 * h + r8) * 4u,
                                (uint32_t)s ^ ((uint32_t)(s >> 31) | 0x80000000u));
        }
      }
      float a[2] = {1.f, 1.f};                              // of the rows of mt
      const bool moved = f_sync_or(pass);
      if (moved) {
        auto decode = [](uint32_t u) {
          return __uint_as_float(u & 0x80000000u ? u ^ 0x80000000u : ~u);
        };
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const uint32_t u = ptx::ld_shared_u32_volatile(top + (uint32_t)(hb + 8 * h + r8) * 4u);
          if (u != 0u) {
            const float tv = ceilf(decode(u)), f = ptx::ex2(m[h] - tv);   // 0 from -inf
            sum[h] = ptx::f2_mul(sum[h], ptx::f2_pack(f, f));
            m[h] = tv;
          }
        }
#pragma unroll
        for (int k = 0; k < (kR == 64 ? 2 : 1); ++k) {
          const uint32_t u = ptx::ld_shared_u32_volatile(top + (uint32_t)(lane % kR + 32 * k) * 4u);
          if (u != 0u) {
            const float tv = ceilf(decode(u));
            a[k] = ptx::ex2(mt[k] - tv);
            mt[k] = tv;
          }
        }
      }
      const uint32_t sf_base = x.sbase + S::kSfb + wb * 512u;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int row = hb + 8 * h + r8;
        const uint64_t f2 = ptx::f2_pack(fac[h], fac[h]);
#pragma unroll
        for (int k = 1; k < 32 / S::kTok; ++k)              // the other warps of the block
          z[h] = fmaxf(z[h], __uint_as_float(ptx::ld_shared_u32_volatile(
                                 blk + (uint32_t)((slice ^ k) * kR + row) * 4u)));
        // the block exponent, relative to the reference
        const float ref = m[h] == -INFINITY ? 0.f : m[h];
        const float d = fmaxf(ceilf(z[h]) - ref, (float)kBlockMin);
        const uint32_t eb = (uint32_t)(__float2int_rn(d) + 127);
        const float neg = kTarget - ref - d;
        const uint64_t n2 = ptx::f2_pack(neg, neg);
        if (cq == 0) {
          // the row's scale bytes of the block: hi and lo
          const uint32_t at = sf_base + (uint32_t)(tok0 >> 5);
          if (kR == 64) {                                   // bytes: hi, hi, lo, lo
            const uint32_t cell = at + (uint32_t)(row & 31) * 16u + (uint32_t)(row >> 5) * 4u;
            ptx::st_shared_u8(cell, eb);
            ptx::st_shared_u8(cell + 2u, eb);
          } else if (tok0 % 32 == 0) {                      // row r hi, R + r lo
            const int lo_row = kR + row;
            ptx::st_shared_u8(at + (uint32_t)row * 16u, eb);
            ptx::st_shared_u8(at + (uint32_t)(lo_row & 31) * 16u + (uint32_t)(lo_row >> 5) * 4u,
                              eb);
          }
        }
        uint64_t part = 0;                                  // sums over even and odd tokens
        auto one = [&](auto jt) {
          constexpr int j = decltype(jt)::value;
          float e0, e1, w0, w1;
          ptx::f2_unpack(ptx::f2_fma(v[h][j], f2, n2), e0, e1);
          const uint64_t e2 = ptx::f2_pack(ptx::ex2(e0), ptx::ex2(e1));
          part = ptx::f2_add(part, e2);
          ptx::f2_unpack(ptx::f2_mul(e2, sc[j]), w0, w1);
          uint32_t hi, lo;
          f_split(w0, w1, hi, lo);
          constexpr int kByte = 8 * (j & 1);
          if constexpr (S::kWide) {                         // 64-byte rows, lo R rows further
            const uint32_t at = w_at[j >> 1] + wb * S::kWBytes + (uint32_t)h * 512u;
            ptx::st_shared_u16<kByte>(at, (uint16_t)hi);
            ptx::st_shared_u16<kByte + kR * 64>(at, (uint16_t)lo);
          } else {                                          // 128-byte rows, lo behind hi
            const uint32_t at = wb * S::kWBytes + (uint32_t)h * 1024u;
            ptx::st_shared_u16<kByte>(w_at[j >> 1] + at, (uint16_t)hi);
            ptx::st_shared_u16<kByte>((w_at[j >> 1] ^ 64u) + at, (uint16_t)lo);
          }
        };
        one(std::integral_constant<int, 0>{});
        if constexpr (kJ > 1) one(std::integral_constant<int, 1>{});
        if constexpr (kJ > 2) {
          one(std::integral_constant<int, 2>{});
          one(std::integral_constant<int, 3>{});
        }
        const float bs = __uint_as_float((eb - (uint32_t)kSumShift) << 23);
        sum[h] = ptx::f2_fma(part, ptx::f2_pack(bs, bs), sum[h]);
      }
      ptx::fence_proxy_async_smem();
      if (moved && pg > pb) {
        // O^T's columns, after the P.V of page g - 1 (this page's waits for us)
        f_wait(x, x.bar(F_PEMPTY + (wb ^ 1u)), ((g - 1) >> 1) & 1u);
        __syncwarp();
        ptx::tc_fence_after();
        f_rescale<kR>(x.tmem + lanes + S::kColO + 2u * S::kCols * (uint32_t)grp, a[0], a[1]);
      }
      ptx::tc_fence_before();
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(x.bar(F_PFULL + wb));
      top_i = top_i == 2 ? 0 : top_i + 1;
      stg = stg == kFStages - 1 ? 0 : stg + 1;
    }
    // the next entry's Q (its first score MMA then overlaps this epilogue)
    int nb = 0, npb = 0, npe = 0;
    const bool nhave = it.next(nb, npb, npe);
    if (nhave) load_q(nb);

    // ---- sums, lse, and O / sum ----
    if (!slot_ok && tid == 0) atomicCAS(x.err, 0, MLA_ERR_PLAN);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      float s0, s1;
      ptx::f2_unpack(sum[h], s0, s1);
      s0 += s1;
      s0 += __shfl_xor_sync(0xffffffffu, s0, 1);
      s0 += __shfl_xor_sync(0xffffffffu, s0, 2);
      if (cq == 0)
        ptx::st_shared_u32(x.sbase + S::kSum + (uint32_t)(slice * kR + hb + 8 * h + r8) * 4u,
                           __float_as_uint(s0));
    }
    f_sync();
    if (slice < 2 && cq == 0) {   // the factors, and beside them the lse
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int row = hb + 8 * h + r8;
        float tot = 0.f;
#pragma unroll
        for (int k = 0; k < S::kSlices; ++k)
          tot += __uint_as_float(
              ptx::ld_shared_u32_volatile(x.sbase + S::kSum + (uint32_t)(k * kR + row) * 4u));
        if (slice == 0)
          ptx::st_shared_u32(x.sbase + S::kFac + (uint32_t)row * 4u,
                             __float_as_uint(tot == 0.f ? 0.f : 1.0f / tot));
        else if (row < n_rows && slot_ok) {
          // unshifted where that stays finite: the logarithm has more bits there
          const float l2 = tot < kTotShift ? log2f(tot * kTotShift)
                                           : log2f(tot) + (float)kSumShift;   // NaN too
          *lse_at[h] = tot == 0.f ? -INFINITY : (m[h] - kTarget + l2) * kFLn2;
        }
      }
    }
    // every P.V of the entry is done once the last page's is
    f_wait(x, x.bar(F_PEMPTY + ((g - 1) & 1u)), ((g - 1) >> 1) & 1u);
    __syncwarp();
    ptx::tc_fence_after();
    f_sync();
    const int64_t row0 = (int64_t)b * prm.s_q * prm.h_q + w.tile * kF8TileRows;
    constexpr int kRC = kR < 32 ? kR : 32;                  // rows handled together
#pragma unroll 1
    for (int ch = 0; ch < 2 * (kR / kRC); ++ch) {           // this group's two blocks
      const int mb = 2 * grp + ch / (kR / kRC), r0 = (ch % (kR / kRC)) * kRC;
      const int d = 128 * mb + tl;                          // this lane's dim
      float val[kRC];
      {
        uint32_t o[32];
        ptx::tmem_ld32_wait(x.tmem + lanes + S::kColO + S::kCols * (uint32_t)mb + (uint32_t)r0, o);
        if constexpr (kR == 32) {
          uint32_t lo[32];
          ptx::tmem_ld32_wait(x.tmem + lanes + S::kColO + S::kCols * (uint32_t)mb + 32u, lo);
#pragma unroll
          for (int j = 0; j < kRC; ++j)
            val[j] = __uint_as_float(o[j]) + __uint_as_float(lo[j]);
        } else if constexpr (kR == 16) {
#pragma unroll
          for (int j = 0; j < kRC; ++j)
            val[j] = __uint_as_float(o[j]) + __uint_as_float(o[16 + j]);
        } else {
#pragma unroll
          for (int j = 0; j < kRC; ++j) val[j] = __uint_as_float(o[j]);
        }
      }
#pragma unroll
      for (int j = 0; j < kRC; j += 4) {
        const uint4 f = ptx::ld_shared_v4u(x.sbase + S::kFac + (uint32_t)(r0 + j) * 4u);
        const float fv[4] = {__uint_as_float(f.x), __uint_as_float(f.y), __uint_as_float(f.z),
                             __uint_as_float(f.w)};
#pragma unroll
        for (int k = 0; k < 4; ++k) val[j + k] = fv[k] == 0.f ? 0.f : val[j + k] * fv[k];
      }
      if (!direct) {
        // partials: [slot][row / 4][dim][4 rows]
        if (slot_ok) {
          float4* dst = reinterpret_cast<float4*>(prm.ws_o) +
                        (slot * (kR / 4) + r0 / 4) * kDv + d;
#pragma unroll
          for (int j = 0; j < kRC; j += 4)
            dst[(int64_t)(j / 4) * kDv] = make_float4(val[j], val[j + 1], val[j + 2], val[j + 3]);
        }
      } else if (prm.out_f32) {
        float* dst = static_cast<float*>(prm.out) + (row0 + r0) * kDv + d;
#pragma unroll
        for (int j = 0; j < kRC; ++j)
          if (r0 + j < n_rows) dst[(int64_t)j * kDv] = val[j];
      } else {
        // neighbouring lanes swap so that each stores two dims of one row
        const int odd = lane & 1;
        uint32_t* dst = reinterpret_cast<uint32_t*>(
            static_cast<__nv_bfloat16*>(prm.out) + (row0 + r0 + odd) * kDv + (d & ~1));
#pragma unroll
        for (int j = 0; j < kRC; j += 2) {
          const float give = odd ? val[j] : val[j + 1];
          const float got = __shfl_xor_sync(0xffffffffu, give, 1);
          const uint32_t pk = odd ? ptx::pack_bf16x2(got, val[j + 1]) : ptx::pack_bf16x2(val[j], got);
          if (r0 + j + odd < n_rows) dst[(int64_t)j * (kDv / 2)] = pk;
        }
      }
    }
    ptx::tc_fence_before();
    // the tables are written anew only after the next barrier, which every
    // warp reaches after its reads here
    ++n_item;
    b = nb;
    pb = npb;
    pe = npe;
    have = nhave;
  }
}

template <int kR>
__global__ void __launch_bounds__(kFThreads, 1)
    mla_decode_fp8_kernel(const __grid_constant__ CUtensorMap tm_lat,
                          const __grid_constant__ CUtensorMap tm_rope, const Fp8Params prm) {
  using S = FShape<kR>;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  FCtx x;
  x.sbase = (ptx::smem_addr(smem_raw) + 1023u) & ~1023u;
  x.bar0 = x.sbase + S::kBar;
  x.abort_addr = x.sbase + S::kMisc + 4;
  x.err = prm.err;
  const uint32_t tmem_slot = x.sbase + S::kMisc;

  if (threadIdx.x == 0) {
    for (int s = 0; s < kFStages; ++s) {
      ptx::mbar_init(x.bar(F_FULL + s), 2);
      ptx::mbar_init(x.bar(F_EMPTY + s), 1);
    }
    for (int s = 0; s < 2; ++s) {
      ptx::mbar_init(x.bar(F_SFULL + s), 2);
      ptx::mbar_init(x.bar(F_SEMPTY + s), kFSoftWarps);
      ptx::mbar_init(x.bar(F_PFULL + s), kFSoftWarps);
      ptx::mbar_init(x.bar(F_PEMPTY + s), 1);
    }
    ptx::mbar_init(x.bar(F_QFULL), kFSoftWarps);
    ptx::mbar_init(x.bar(F_QEMPTY), 1);
    ptx::mbar_init(x.bar(F_TEARDOWN), 2);   // both issuing warps
    ptx::st_shared_u32(x.abort_addr, 0u);
    ptx::fence_mbarrier_init();
  }
  if (warp == kFMmaWarp) {
    ptx::tmem_alloc(tmem_slot, kFTmemCols);
    ptx::tmem_relinquish();
  }
  if (warp == kFProducerWarp && lane == 0) {
    ptx::prefetch_tmap(&tm_lat);
    ptx::prefetch_tmap(&tm_rope);
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  x.tmem = ptx::ld_shared_u32_volatile(tmem_slot);

  // While an earlier kernel still runs, the queries come into L2 (a line a
  // thread, where that covers them: ragged batch of 64, cold: 93.0 -> 90.7 us).
  // A line written meanwhile is written in L2, so the loads below see it.
  {
    const int64_t line = (int64_t)blockIdx.x * kFThreads + threadIdx.x;
    if (line < (int64_t)prm.batch * prm.s_q * prm.h_q * (kDqk * 2) / 128)
      ptx::prefetch_l2(static_cast<const char*>(prm.q) + line * 128);
  }
  // The plan (and the inputs) come from earlier kernels on the stream.
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  // The plan must describe this call.  The header first (two words a load): a
  // plan of another shape may end before this CTA's entry.
  const int32_t* plan = prm.plan;
  FWork w = {};
  bool has_work = false;
  const int tiles = f8_tiles(prm.s_q, prm.h_q), gt = prm.workers / tiles;
  const int tile = (int)blockIdx.x % tiles, c = (int)blockIdx.x / tiles;
  const int2* h2 = reinterpret_cast<const int2*>(plan);
  const int2 h01 = h2[0], h23 = h2[1], h45 = h2[2], h67 = h2[3], h89 = h2[4];
  static_assert(H_MAGIC == 0 && H_BATCH == 1 && H_SQ == 2 && H_HQ == 3 && H_TILES == 4 &&
                    H_GT == 5 && H_GUSED == 6 && H_STOTAL == 7 && H_NCLUSTERS == 9,
                "the header's words, two a load");
  const bool ours = (h01.x == kF8PlanMagic) & (h01.y == prm.batch) & (h23.x == prm.s_q) &
                    (h23.y == prm.h_q) & (h45.x == tiles) & (h45.y == gt) & (h89.y == prm.workers);
  w.tile = tile;
  w.stotal = h67.y;
  w.items = plan + plan_off_items(gt) / 4;
  bool bad = !ours;
  if (ours && c < h67.x) {
    const int2* e = reinterpret_cast<const int2*>(plan + H_WORDS + c * kClusterWords);
    const int2 e01 = e[0], e23 = e[1], e45 = e[2];
    w.b0 = e01.x;
    w.p0 = e01.y;
    w.b1 = e23.x;
    w.p1 = e23.y;
    w.split0 = e45.x;
    bad = w.b0 < 0 || w.p0 < 0 || w.p1 < 0 || w.b0 > w.b1 || w.b1 > prm.batch ||
          (w.b1 == prm.batch && w.p1 != 0);
    has_work = !bad && !(w.b0 == w.b1 && w.p0 >= w.p1);
  }
  if (bad && threadIdx.x == 0) atomicCAS(prm.err, 0, MLA_ERR_PLAN);

  if (!has_work) {
    // nothing to do: fall through to the teardown
  } else if (warp == kFProducerWarp) {
    if (lane == 0) f_producer(x, w, prm, &tm_lat, &tm_rope, tiles == 1);
  } else if (warp == kFMmaWarp) {
    f_mma_s<kR>(x, w, lane);   // whole warp: one elected lane issues
  } else if (warp == kFPvWarp) {
    f_mma_o<kR>(x, w);
  } else if (warp == kFScaleWarp) {
    f_scales<kR>(x, w, prm, lane);
  } else {
    f_softmax<kR>(x, w, prm, warp, lane);
  }
  __syncwarp();

  // Teardown.  After an abort, give in-flight copies and MMAs time to land
  // before the shared memory and TMEM are released.
  if (warp == kFMmaWarp || warp == kFPvWarp) {
    ptx::mma_commit_elect(x.bar(F_TEARDOWN));   // this warp's MMAs are done
    const uint64_t t0 = ptx::globaltimer();
    while (!ptx::mbar_try_wait(x.bar(F_TEARDOWN), 0u)) {
      if (ptx::globaltimer() - t0 > kFWaitNs) {
        if (lane == 0) atomicCAS(x.err, 0, MLA_ERR_DEVICE_TIMEOUT);
        break;
      }
    }
  }
  if (ptx::ld_shared_u32_volatile(x.abort_addr) != 0u) {
    const uint64_t t0 = ptx::globaltimer();
    while (ptx::globaltimer() - t0 < kFDrainNs) __nanosleep(1000);
  }
  __syncwarp();
  ptx::tc_fence_before();
  __syncthreads();
  if (warp == kFMmaWarp) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc(x.tmem, kFTmemCols);
  }
}

// ------------------------------------------------------------------ combine
// Merges the partials of every (entry, tile) with two or more splits:
//   lse = m + ln(sum_j exp(lse_j - m)),  out = sum_j exp(lse_j - m) o_j / sum
// Each CTA first lists the entries that need it (one load a thread for 128
// entries), then takes jobs of four rows and one of `parts` ranges of the
// dims; a float4 holds the four rows of one dim and split.  Two dims and four
// splits of each are loaded together (with one part four dims and two splits:
// where there are many jobs an entry has few splits), the first of them while
// the warp turns the splits' lse into weights (lane 4 j + k: row k of splits j,
// j + 8, ...) in its own part of shared memory; no warp waits for another.  With
// eight parts a warp has all the job's 64 dims, and the warps (four, or 16 for
// many splits) share the splits, turn them into weights together and add up at
// the end.  What bounds it is latency: the chain of a job
// (list, lse, weights, sums) and the fetch of its code, which is why the loops
// are rolled and each number of parts has a kernel (one for all: 16 x 128 heads
// over 4096 tokens 29.95 us against 29.2, plan and decode).  So there are as
// many parts as still have all jobs on the SMs at once (that call: 512 jobs of
// one part 30.3 us a decode, 1024 of two 27.3; 8 x 16 heads over 65536 tokens:
// 128 jobs whose warps split the dims 54.0, 256 whose warps share 19 splits
// 52.3; ragged batch of 64, one part: two dims a load 75.7, four 73.2), and
// registers for seven CTAs an SM (eight spilled: that batch 76.1 against 74.5).
// Entries without pages get out = 0, lse = -inf.
constexpr int kF8CombineCtas = 7;   // an SM
constexpr int kF8ShareParts = 8;    // with so many the warps share the splits
constexpr int kF8WidePages = 15;    // least shares a table holds from which they may be 16
constexpr int kF8MaxSplits = 256;   // an entry has at most as many splits as a tile's CTAs

template <int parts, int kWarps>
__global__ void __launch_bounds__(32 * kWarps, kWarps == 16 ? 2 : parts == 1 ? 6 : kF8CombineCtas)
    mla_fp8_combine_kernel(const Fp8Params p, const int rows_t) {
  constexpr int kThreads = 32 * kWarps;
  constexpr int kC = parts == 1 ? 4 : 2, kJ = 8 / kC;       // dims and splits a load
  constexpr bool share = parts == kF8ShareParts;
  constexpr int dims = kDv / parts;                         // of a job
  constexpr int dstep = share ? 32 : kThreads;              // between a thread's dims
  __shared__ int s_list[3][kThreads];                       // entry, splits, first slot
  __shared__ int s_warp[kWarps];
  __shared__ __align__(16) float s_w[share ? 1 : kWarps][4 * kF8MaxSplits];
  __shared__ float s_red[2][kWarps][4];                     // maxima and sums of the warps' splits
  __shared__ float4 s_acc[share ? kWarps : 1][kC][32];
  // The plan is read before the wait: the main kernel lets this grid launch
  // only after its own wait on the planner had returned.
  bool waited = false;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int rows = p.s_q * p.h_q;
  const int tiles = f8_tiles(p.s_q, p.h_q), gt = p.workers / tiles;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int32_t* items = p.plan + plan_off_items(gt) / 4;
  // A plan of another call may end before its items: the main kernel reports
  // it, and the outputs stay as they are.
  const int head = f_plan_head(p.plan, lane);
  const int stotal = __shfl_sync(0xffffffffu, head, H_STOTAL);
  const int entries = f_plan_ours(head, p, lane) ? p.batch : 0;
  const int groups = rows_t / 4;                            // of four rows in a tile
  const int j_first = share ? kJ * warp : 0, j_step = share ? kJ * kWarps : kJ;
  float* sw = s_w[share ? 0 : warp];
  for (int base = 0; base < entries; base += kThreads) {
    const int mine = base + (int)threadIdx.x;
    const int splits = mine < p.batch ? __ldcg(items + mine * kItemWords + 1) : 1;
    const int first = mine < p.batch ? __ldcg(items + mine * kItemWords + 2) : 0;
    const unsigned bal = __ballot_sync(0xffffffffu, splits != 1);
    __syncthreads();                                        // the last list is read
    if (lane == 0) s_warp[warp] = __popc(bal);
    __syncthreads();
    int before = 0, count = 0;
#pragma unroll
    for (int k = 0; k < kWarps; ++k) {
      before += k < warp ? s_warp[k] : 0;
      count += s_warp[k];
    }
    if (splits != 1) {
      const int at = before + __popc(bal & ((1u << lane) - 1u));
      s_list[0][at] = mine;
      s_list[1][at] = splits;
      s_list[2][at] = first;
    }
    __syncthreads();
    const int jobs = count * tiles * groups * parts;
#pragma unroll 1
    for (int job = (int)blockIdx.x; job < jobs; job += (int)gridDim.x) {
      const int q = job / parts, part = job - q * parts, at = q / (groups * tiles);
      const int rg = q % groups, tile = q / groups % tiles;
      const int b = s_list[0][at], ns = s_list[1][at];
      const int r0 = tile * kF8TileRows + 4 * rg;           // first row within the entry
      if (r0 >= rows) continue;
      const int64_t slot0 = (int64_t)tile * stotal + s_list[2][at];
      if (ns < 0 || ns > kF8MaxSplits ||
          (ns > 1 && (slot0 < 0 || slot0 + ns > f8_slots(p.workers)))) {
        if (threadIdx.x == 0) atomicCAS(p.err, 0, MLA_ERR_PLAN);
        continue;
      }
      if (!waited) {
        asm volatile("griddepcontrol.wait;" ::: "memory");
        waited = true;
      }
      const int d0 = part * dims + (share ? lane : (int)threadIdx.x);
      const float4* o_col =
          reinterpret_cast<const float4*>(p.ws_o) + (slot0 * groups + rg) * kDv + d0;
      const int step = groups * kDv;
      float4 v[kJ][kC];
      auto load = [&](int d, int j0) {
        const float4* src = o_col + (int64_t)j0 * step + d;
#pragma unroll
        for (int j = 0; j < kJ; ++j)
#pragma unroll
          for (int c = 0; c < kC; ++c)
            v[j][c] = j0 + j < ns ? __ldcs(src + j * step + c * dstep)
                                  : make_float4(0.f, 0.f, 0.f, 0.f);
      };
      load(0, j_first);
      const float* lse_col = p.ws_lse + slot0 * rows_t + 4 * rg + (lane & 3);
      // a warp has all the splits' weights, or a share of them where the warps
      // share the splits
      const int j_mine = share ? (int)threadIdx.x >> 2 : lane >> 2;
      constexpr int kStride = share ? kThreads / 4 : 8;
      float m = -INFINITY, se = 0.f;
#pragma unroll 1
      for (int j = j_mine; j < ns; j += kStride) {
        const float y = __ldcs(lse_col + j * rows_t);
        sw[4 * j + (lane & 3)] = y;
        m = fmaxf(m, y);
      }
#pragma unroll
      for (int o = 4; o < 32; o <<= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
      if constexpr (share) {
        if (lane < 4) s_red[0][warp][lane] = m;
        __syncthreads();
#pragma unroll
        for (int k = 0; k < kWarps; ++k) m = fmaxf(m, s_red[0][k][lane & 3]);
      }
#pragma unroll 1
      for (int j = j_mine; j < ns; j += kStride) {
        const float y = sw[4 * j + (lane & 3)];
        const float e = y == -INFINITY ? 0.f : expf(y - m);   // a NaN stays one
        sw[4 * j + (lane & 3)] = e;
        se += e;
      }
#pragma unroll
      for (int o = 4; o < 32; o <<= 1) se += __shfl_xor_sync(0xffffffffu, se, o);
      if constexpr (share) {
        if (lane < 4) s_red[1][warp][lane] = se;
        __syncthreads();                                    // the weights too
        se = 0.f;
#pragma unroll
        for (int k = 0; k < kWarps; ++k) se += s_red[1][k][lane & 3];
      }
      if (threadIdx.x < 4 && r0 + lane < rows && part == 0) {
        const int row = r0 + lane, qi = row / p.h_q, h = row - qi * p.h_q;
        p.lse[((int64_t)b * p.h_q + h) * p.s_q + qi] = se == 0.f ? -INFINITY : m + logf(se);
      }
      const float inv = se == 0.f ? 0.f : 1.0f / se;
      __syncwarp();
#pragma unroll 1
      for (int d = 0; d < dims; d += kC * dstep) {
        float acc[kC][4] = {};
#pragma unroll 1
        for (int j0 = j_first; j0 < ns; j0 += j_step) {
          if (d > 0 || j0 > j_first) load(d, j0);
#pragma unroll
          for (int j = 0; j < kJ; ++j) {
            if (j0 + j >= ns) break;
            const float4 w = *reinterpret_cast<const float4*>(sw + 4 * (j0 + j));
#pragma unroll
            for (int c = 0; c < kC; ++c) {
              acc[c][0] += w.x * v[j][c].x;
              acc[c][1] += w.y * v[j][c].y;
              acc[c][2] += w.z * v[j][c].z;
              acc[c][3] += w.w * v[j][c].w;
            }
          }
        }
        if constexpr (share) {
#pragma unroll
          for (int c = 0; c < kC; ++c)
            s_acc[warp][c][lane] = make_float4(acc[c][0], acc[c][1], acc[c][2], acc[c][3]);
          __syncthreads();
          if (warp > 0) continue;   // to the barrier at the job's end
#pragma unroll
          for (int c = 0; c < kC; ++c)
#pragma unroll
            for (int k = 1; k < kWarps; ++k) {
              const float4 o = s_acc[k][c][lane];
              acc[c][0] += o.x;
              acc[c][1] += o.y;
              acc[c][2] += o.z;
              acc[c][3] += o.w;
            }
        }
        const int64_t o0 = ((int64_t)b * rows + r0) * kDv + d0 + d;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const float f = __shfl_sync(0xffffffffu, inv, k);
          if (r0 + k < rows) {
#pragma unroll
            for (int c = 0; c < kC; ++c) {
              const int64_t o = o0 + k * kDv + c * dstep;
              if (p.out_f32)
                static_cast<float*>(p.out)[o] = acc[c][k] * f;
              else
                static_cast<__nv_bfloat16*>(p.out)[o] = __float2bfloat16_rn(acc[c][k] * f);
            }
          }
        }
      }
      // the weights (and sums) are read
      if constexpr (share)
        __syncthreads();
      else
        __syncwarp();
    }
  }
  // every block waits once, so that this grid completes only after the main one
  if (!waited) asm volatile("griddepcontrol.wait;" ::: "memory");
}

constexpr int kMaxFp8Devices = 64;
std::once_flag g_fp8_once[kMaxFp8Devices];
cudaError_t g_fp8_status[kMaxFp8Devices];

template <int kR>
cudaError_t f8_attr() {
  return cudaFuncSetAttribute(mla_decode_fp8_kernel<kR>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                              (int)FShape<kR>::kSmemAlloc);
}

}  // namespace

cudaError_t launch_decode_fp8(const CUtensorMap& kv_lat, const CUtensorMap& kv_rope,
                              const Fp8Params& p, int num_sms, cudaStream_t stream) {
  int device = 0;
  cudaError_t e = cudaGetDevice(&device);
  if (e != cudaSuccess) return e;
  if (device < 0 || device >= kMaxFp8Devices) return cudaErrorInvalidDevice;
  std::call_once(g_fp8_once[device], [&]() {
    cudaError_t s = f8_attr<16>();
    if (s == cudaSuccess) s = f8_attr<32>();
    if (s == cudaSuccess) s = f8_attr<64>();
    g_fp8_status[device] = s;
  });
  if (g_fp8_status[device] != cudaSuccess) return g_fp8_status[device];

  const int tiles = f8_tiles(p.s_q, p.h_q), rows_t = f8_rows(p.s_q, p.h_q);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(p.workers / tiles * tiles);
  cfg.blockDim = dim3(kFThreads);
  cfg.dynamicSmemBytes = rows_t == 16   ? FShape<16>::kSmemAlloc
                         : rows_t == 32 ? FShape<32>::kSmemAlloc
                                        : FShape<64>::kSmemAlloc;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  e = rows_t == 16   ? cudaLaunchKernelEx(&cfg, mla_decode_fp8_kernel<16>, kv_lat, kv_rope, p)
      : rows_t == 32 ? cudaLaunchKernelEx(&cfg, mla_decode_fp8_kernel<32>, kv_lat, kv_rope, p)
                     : cudaLaunchKernelEx(&cfg, mla_decode_fp8_kernel<64>, kv_lat, kv_rope, p);
  if (e != cudaSuccess) return e;
  // As many parts as still have all jobs on the SMs at once.  Where the warps
  // share the splits and an entry may have 16 or more (from the workers and the
  // pages of the block table), 16 warps: one entry of 20000 tokens with 64 heads
  // 32.9 -> 21.0 us, of 4096 with 16 heads 14.2 -> 13.3; with fewer splits they
  // only start later (four entries of up to 300 tokens, 32 heads 13.4 -> 14.4,
  // which a table as wide as a context limit costs such a batch).
  // The table's width reaches no bit of the results: an entry that it bounds to
  // fewer than kF8WidePages least shares has at most 16 splits (P pages touch at
  // most (P - 1 + m - 1) / m + 1 workers of m units or more), and those both forms
  // add up in the same order, four a warp.
  const int64_t quads = (int64_t)p.batch * tiles * (rows_t / 4);
  const int64_t cap = kF8CombineCtas * (int64_t)num_sms;
  const int parts = quads * kF8ShareParts <= cap ? kF8ShareParts : quads * 2 <= cap ? 2 : 1;
  const int64_t jobs = quads * parts;
  const bool wide = parts == kF8ShareParts && jobs <= 2 * (int64_t)num_sms &&
                    p.workers / tiles / p.batch >= 16 &&
                    p.max_pages / f8_min_units(rows_t) >= kF8WidePages;
  cfg.gridDim = dim3((unsigned)(jobs < cap ? jobs : cap));
  cfg.blockDim = dim3(wide ? 512 : 128);
  cfg.dynamicSmemBytes = 0;
  return wide         ? cudaLaunchKernelEx(&cfg, mla_fp8_combine_kernel<kF8ShareParts, 16>, p, rows_t)
         : parts == 1 ? cudaLaunchKernelEx(&cfg, mla_fp8_combine_kernel<1, 4>, p, rows_t)
         : parts == 2 ? cudaLaunchKernelEx(&cfg, mla_fp8_combine_kernel<2, 4>, p, rows_t)
                      : cudaLaunchKernelEx(&cfg, mla_fp8_combine_kernel<kF8ShareParts, 4>, p, rows_t);
}

}  // namespace mla
