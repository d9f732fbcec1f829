// Cache append with the rotary position embedding applied on the way, into
// bf16 pages (mla_rope_append) or into e4m3 pages with one fp32 scale for
// each block of G tokens (mla_rope_append_fp8).
//
// Mathematics.  Pair j (j < 32) of a token's 64 rotary dims at position t is
// turned by the angle whose cosine and sine are table[t][j], table[t][32+j]:
//   y0 = x0 c - x1 s,   y1 = x1 c + x0 s       (fp32, rounded once on store)
// The pairs are the dims (2j, 2j+1) or (j, 32+j).  The 512 latent dims pass
// unturned.  The 8-bit form stores e4m3(x / scale), scale = amax / 448 over the
// block's new rows, at least 2^-100 (the reciprocal stays finite) and at least
// the scale that the block's earlier tokens were stored with; where that makes
// the scale grow, the earlier rows of the block are stored anew as
// e4m3(code * (old / scale)).  Between bf16 numbers x 448 / amax is often just
// half way between two codes, so it is not taken from the rounded scale: with
// 448 / amax = hi + lo (two fp32 numbers) the fused x hi + (x lo) is the fp32
// number nearest to the quotient, half way where the quotient is.
//
// What bounds it: memory.  A token moves 1152 bytes in and 1152 (bf16) or 576
// + 4 / G out, a (token, head) of the queries 128 in and 128 out; with 128
// heads the queries are nine tenths of it.  4096 tokens with 128 heads take
// 25.5 us in either form (5.7 and 5.6 TB/s).  A call with few tokens is one
// launch and a chain of four loads (length, table, angles, rows): calls one
// after the other in a graph take 2.2 us for one token, 3.9 for 264 tokens with
// 128 heads and scales of 16.
// The rows and the queries are one grid, so that neither waits for the other.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "mla.h"
#include "mla_internal.h"

namespace mla {
namespace {

constexpr int kRopeThreads = 256;
constexpr int kRopeWarps = kRopeThreads / 32;
constexpr int kRopeDims = kDqk - kDv;        // 64
constexpr int kRopePairs = kRopeDims / 2;    // 32
constexpr int kQHeads = kRopeThreads / 8;    // heads a CTA turns in one step (8 threads each)
constexpr float kE4m3Max = 448.0f;
constexpr float kScaleMin = 7.8886090522101181e-31f;   // 2^-100

struct RopeArgs {
  const __nv_bfloat16* kv_new;
  int64_t kv_sb, kv_ss;                    // strides in elements: batch, token
  const __nv_bfloat16* q_in;
  __nv_bfloat16* q_out;
  int64_t qi_sb, qi_ss, qi_sh, qo_sb, qo_ss, qo_sh;   // batch, token, head
  void* cache;
  float* scales;
  int num_pages, max_pages;
  const int32_t* block_table;
  const int32_t* seqlens;
  const int32_t* new_lens;                 // null: s_new for every entry
  const float* cos_sin;
  int max_pos, interleaved;
  int batch, s_new, h_q;
  int chunks;                              // append CTAs per batch entry
  int head_steps;                          // CTAs per token of the query part
  int heads_per_thread;                    // 1 or 4
  int64_t append_ctas;
  int* err;
};

// The entry's first new position and its count of new tokens; -1 tokens when
// the count is out of range.
__device__ __forceinline__ void rope_entry(const RopeArgs& a, int b, int& start, int& n) {
  const int L = max(a.seqlens[b], -(1 << 30));              // any negative one is as bad
  n = a.new_lens ? a.new_lens[b] : a.s_new;
  if (n < 0 || n > a.s_new) n = -1;
  start = L - (n > 0 ? n : 0);
}

__device__ __forceinline__ bool rope_pos_ok(const RopeArgs& a, int t) {
  return t >= 0 && t < a.max_pos && (int64_t)t < (int64_t)a.max_pages * kPageTokens;
}

// Pool row of position t of entry b, or -1 when its page is outside the pool.
__device__ __forceinline__ int64_t rope_row(const RopeArgs& a, int b, int t) {
  const int page = a.block_table[(int64_t)b * a.max_pages + t / kPageTokens];
  if ((unsigned)page >= (unsigned)a.num_pages) return -1;
  return (int64_t)page * kPageTokens + t % kPageTokens;
}

__device__ __forceinline__ float2 bf2(uint32_t u) {
  return make_float2(__uint_as_float(u << 16), __uint_as_float(u & 0xffff0000u));
}
__device__ __forceinline__ uint32_t pack_bf(float lo, float hi) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}
__device__ __forceinline__ uint32_t pack_e4m3(float lo, float hi) {
  return __nv_cvt_float2_to_fp8x2(make_float2(lo, hi), __NV_SATFINITE, __NV_E4M3);
}

// Pair `lane` of a row's rotary dims, turned.
__device__ __forceinline__ float2 rope_pair(const RopeArgs& a, const __nv_bfloat16* x, int t,
                                            int lane) {
  float x0, x1;
  if (a.interleaved) {
    const float2 v = bf2(*reinterpret_cast<const uint32_t*>(x + 2 * lane));
    x0 = v.x;
    x1 = v.y;
  } else {
    x0 = __bfloat162float(x[lane]);
    x1 = __bfloat162float(x[lane + kRopePairs]);
  }
  const float* cs = a.cos_sin + (int64_t)t * kRopeDims;
  const float c = cs[lane], s = cs[kRopePairs + lane];
  return make_float2(x0 * c - x1 * s, x1 * c + x0 * s);
}

// Query part: CTA k of the part turns heads_per_cta heads of one token, eight
// threads to a head (thread j the pairs 4j .. 4j + 3), HPT heads a thread.  The
// queries do not depend on the lengths, so they are loaded first and the
// position and its angles arrive meanwhile.
template <int HPT>
__device__ __forceinline__ void rope_queries(const RopeArgs& a, int64_t k) {
  const int64_t token = k / a.head_steps;
  const int h0 = (int)(k - token * a.head_steps) * (HPT * kQHeads) + (threadIdx.x >> 3);
  const int b = (int)(token / a.s_new), i = (int)(token - (int64_t)b * a.s_new);
  const int j = threadIdx.x & 7;
  const __nv_bfloat16* src = a.q_in + (int64_t)b * a.qi_sb + (int64_t)i * a.qi_ss;
  uint4 x[HPT];
#pragma unroll
  for (int p = 0; p < HPT; ++p) {
    const int h = h0 + p * kQHeads;
    if (h < a.h_q) {
      const __nv_bfloat16* row = src + (int64_t)h * a.qi_sh;
      if (a.interleaved) {                 // 8 consecutive dims
        x[p] = __ldcs(reinterpret_cast<const uint4*>(row + 8 * j));
      } else {                             // 4 dims of each half
        const uint2 u = __ldcs(reinterpret_cast<const uint2*>(row + 4 * j));
        const uint2 w = __ldcs(reinterpret_cast<const uint2*>(row + kRopePairs + 4 * j));
        x[p] = make_uint4(u.x, u.y, w.x, w.y);
      }
    }
  }
  int start, n;
  rope_entry(a, b, start, n);
  if (i >= n) return;
  const int t = start + i;
  if (!rope_pos_ok(a, t)) return;          // flagged by the append part
  const float4 c4 = *reinterpret_cast<const float4*>(a.cos_sin + (int64_t)t * kRopeDims + 4 * j);
  const float4 s4 =
      *reinterpret_cast<const float4*>(a.cos_sin + (int64_t)t * kRopeDims + kRopePairs + 4 * j);
  const float c[4] = {c4.x, c4.y, c4.z, c4.w}, s[4] = {s4.x, s4.y, s4.z, s4.w};
  __nv_bfloat16* dst = a.q_out + (int64_t)b * a.qo_sb + (int64_t)i * a.qo_ss;
#pragma unroll
  for (int p = 0; p < HPT; ++p) {
    const int h = h0 + p * kQHeads;
    if (h >= a.h_q) break;
    __nv_bfloat16* y = dst + (int64_t)h * a.qo_sh;
    if (a.interleaved) {
      uint32_t w[4] = {x[p].x, x[p].y, x[p].z, x[p].w};
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const float2 f = bf2(w[q]);
        w[q] = pack_bf(f.x * c[q] - f.y * s[q], f.y * c[q] + f.x * s[q]);
      }
      *reinterpret_cast<uint4*>(y + 8 * j) = make_uint4(w[0], w[1], w[2], w[3]);
    } else {
      const float2 p0 = bf2(x[p].x), p1 = bf2(x[p].y), r0 = bf2(x[p].z), r1 = bf2(x[p].w);
      const float x0[4] = {p0.x, p0.y, p1.x, p1.y}, x1[4] = {r0.x, r0.y, r1.x, r1.y};
      float y0[4], y1[4];
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        y0[q] = x0[q] * c[q] - x1[q] * s[q];
        y1[q] = x1[q] * c[q] + x0[q] * s[q];
      }
      *reinterpret_cast<uint2*>(y + 4 * j) =
          make_uint2(pack_bf(y0[0], y0[1]), pack_bf(y0[2], y0[3]));
      *reinterpret_cast<uint2*>(y + kRopePairs + 4 * j) =
          make_uint2(pack_bf(y1[0], y1[1]), pack_bf(y1[2], y1[3]));
    }
  }
}

// One token's row on a warp: 16 latent dims a lane (packed bf16) and the turned
// rotary pair.
struct RopeRow {
  uint4 v[2];
  float2 y;
  __device__ __forceinline__ void load(const RopeArgs& a, int b, int i, int t, int lane) {
    const __nv_bfloat16* src = a.kv_new + (int64_t)b * a.kv_sb + (int64_t)i * a.kv_ss;
    v[0] = reinterpret_cast<const uint4*>(src)[2 * lane];
    v[1] = reinterpret_cast<const uint4*>(src)[2 * lane + 1];
    y = rope_pair(a, src + kDv, t, lane);
  }
  __device__ __forceinline__ float amax() const {
    const uint32_t w[8] = {v[0].x, v[0].y, v[0].z, v[0].w, v[1].x, v[1].y, v[1].z, v[1].w};
    float m = fmaxf(fabsf(y.x), fabsf(y.y));
#pragma unroll
    for (int c = 0; c < 8; ++c) {
      const float2 f = bf2(w[c]);
      m = fmaxf(m, fmaxf(fabsf(f.x), fabsf(f.y)));
    }
    return m;
  }
  // codes of the row times inv.x + inv.y
  __device__ __forceinline__ void store_fp8(const RopeArgs& a, uint8_t* dst, float2 inv,
                                            int lane) const {
    auto over = [inv](float x) { return fmaf(x, inv.x, x * inv.y); };
    const uint32_t w[8] = {v[0].x, v[0].y, v[0].z, v[0].w, v[1].x, v[1].y, v[1].z, v[1].w};
    uint32_t o[4];
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      const float2 f = bf2(w[2 * c]), g = bf2(w[2 * c + 1]);
      o[c] = pack_e4m3(over(f.x), over(f.y)) | (pack_e4m3(over(g.x), over(g.y)) << 16);
    }
    reinterpret_cast<uint4*>(dst)[lane] = make_uint4(o[0], o[1], o[2], o[3]);
    const uint32_t r = pack_e4m3(over(y.x), over(y.y));
    if (a.interleaved) {
      *reinterpret_cast<uint16_t*>(dst + kDv + 2 * lane) = (uint16_t)r;
    } else {
      dst[kDv + lane] = (uint8_t)(r & 0xffu);
      dst[kDv + kRopePairs + lane] = (uint8_t)(r >> 8);
    }
  }
};

// bf16 pages: one warp a token.
template <int HPT>
__global__ void __launch_bounds__(kRopeThreads) mla_rope_append_kernel(const RopeArgs a) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if ((int64_t)blockIdx.x >= a.append_ctas) {
    rope_queries<HPT>(a, (int64_t)blockIdx.x - a.append_ctas);
    return;
  }
  const int b = (int)(blockIdx.x / a.chunks);
  const int i = (int)(blockIdx.x - (int64_t)b * a.chunks) * kRopeWarps + warp;
  int start, n;
  rope_entry(a, b, start, n);
  if (n < 0 && threadIdx.x == 0) atomicCAS(a.err, 0, MLA_ERR_DEVICE_BOUNDS);
  if (i >= n) return;
  const int t = start + i;
  const int64_t row = rope_pos_ok(a, t) ? rope_row(a, b, t) : -1;
  if (row < 0) {
    if (lane == 0) atomicCAS(a.err, 0, MLA_ERR_DEVICE_BOUNDS);
    return;
  }
  const __nv_bfloat16* src = a.kv_new + (int64_t)b * a.kv_sb + (int64_t)i * a.kv_ss;
  __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(a.cache) + row * kDqk;
  const uint4 v0 = reinterpret_cast<const uint4*>(src)[lane];
  const uint4 v1 = reinterpret_cast<const uint4*>(src)[lane + 32];
  const float2 y = rope_pair(a, src + kDv, t, lane);
  reinterpret_cast<uint4*>(dst)[lane] = v0;
  reinterpret_cast<uint4*>(dst)[lane + 32] = v1;
  if (a.interleaved) {
    *reinterpret_cast<uint32_t*>(dst + kDv + 2 * lane) = pack_bf(y.x, y.y);
  } else {
    dst[kDv + lane] = __float2bfloat16_rn(y.x);
    dst[kDv + kRopePairs + lane] = __float2bfloat16_rn(y.y);
  }
}

// e4m3 pages: a CTA takes the new tokens of 8 TPW consecutive positions
// (aligned, so that scale blocks of G tokens lie inside): one block, or 8 / G
// blocks when G < 8.  Warp w takes the TPW tokens from w * TPW; the block's amax
// goes through shared memory.  With more than two tokens a warp the rows are
// read a second time to be stored (they are in L2): holding eight in registers
// took 126 a thread and left too few warps to the query CTAs of the same grid
// (53 against 29 us for 4000 tokens with 128 heads, one scale a page).
template <int TPW, int HPT>
__global__ void __launch_bounds__(kRopeThreads) mla_rope_append_fp8_kernel(const RopeArgs a,
                                                                           const int G) {
  __shared__ float s_amax[kRopeWarps];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if ((int64_t)blockIdx.x >= a.append_ctas) {
    rope_queries<HPT>(a, (int64_t)blockIdx.x - a.append_ctas);
    return;
  }
  constexpr int kSpan = kRopeWarps * TPW;
  constexpr int kHold = TPW < 2 ? TPW : 2;   // rows in registers
  const int b = (int)(blockIdx.x / a.chunks);
  int start, n;
  rope_entry(a, b, start, n);
  if (n < 0 && threadIdx.x == 0) atomicCAS(a.err, 0, MLA_ERR_DEVICE_BOUNDS);
  if (n <= 0) return;
  // floor, so that a negative first position still falls into an aligned span
  const int first = start >= 0 ? start / kSpan : -((-start + kSpan - 1) / kSpan);
  const int base = (first + (int)(blockIdx.x - (int64_t)b * a.chunks)) * kSpan;
  const int end = start + n;
  if (base >= end) return;
  // every position of a span lies in one page (kSpan divides 64)
  const bool span_ok = base >= 0 && (int64_t)base < (int64_t)a.max_pages * kPageTokens;
  const int64_t row0 = span_ok ? rope_row(a, b, base) : -1;
  const int t_lo = base + warp * TPW;      // this warp's positions
  auto have = [&](int t) { return t >= start && t < end && row0 >= 0 && t < a.max_pos; };
  RopeRow row[kHold];
  float amax = -1.f;                       // below any row's, until one is there
#pragma unroll 1
  for (int k0 = 0; k0 < TPW; k0 += kHold) {
#pragma unroll
    for (int k = 0; k < kHold; ++k) {
      const int t = t_lo + k0 + k;
      if (have(t))
        row[k].load(a, b, t - start, t, lane);
      else if (t >= start && t < end && lane == 0)
        atomicCAS(a.err, 0, MLA_ERR_DEVICE_BOUNDS);
    }
#pragma unroll
    for (int k = 0; k < kHold; ++k)
      if (have(t_lo + k0 + k)) amax = fmaxf(amax, row[k].amax());
  }
  // the block of this warp's tokens: warps [w0, w0 + nw) of the CTA
  const int nw = G < kRopeWarps ? G : kRopeWarps;
  const int w0 = warp & ~(nw - 1);
  const int blk = base + w0 * TPW;         // first position of the block
  const int64_t brow = row0 + (blk - base);
  // earlier tokens in the block: their scale, read before anyone replaces it
  const bool held = row0 >= 0 && blk < start && blk + G > start;
  const float old = held ? a.scales[brow / G] : 0.f;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
  if (lane == 0) s_amax[warp] = amax;
  __syncthreads();
  amax = -1.f;
  for (int w = 0; w < nw; ++w) amax = fmaxf(amax, s_amax[w0 + w]);
  if (amax < 0.f) return;                  // no new token of the block is in range
  const float fresh = __fdiv_rn(amax, kE4m3Max);
  float scale = fmaxf(fresh, kScaleMin);
  uint8_t* cache = static_cast<uint8_t*>(a.cache);
  if (held) {
    // the block's scale does not shrink
    scale = fmaxf(scale, old);
    if (scale > old) {
      const float ratio = __fdiv_rn(old, scale);
      for (int r = warp - w0; r < start - blk; r += nw) {
        uint4* p = reinterpret_cast<uint4*>(cache + (brow + r) * kDqk);
        for (int c = lane; c < kDqk / 16; c += 32) {
          const uint4 u = p[c];
          uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            uint32_t r2 = 0;
#pragma unroll
            for (int hf = 0; hf < 2; ++hf) {
              const __half2_raw hr =
                  __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(w[q] >> (16 * hf)), __NV_E4M3);
              const float2 f = __half22float2(__half2(hr));
              r2 |= pack_e4m3(f.x * ratio, f.y * ratio) << (16 * hf);
            }
            w[q] = r2;
          }
          p[c] = make_uint4(w[0], w[1], w[2], w[3]);
        }
      }
    }
  }
  // 448 / amax, or 1 / scale where the scale is another; the remainder over den
  // is its product with the quotient over num
  const bool own = scale == fresh;
  const float num = own ? kE4m3Max : 1.0f, den = own ? amax : scale;
  float2 inv;
  inv.x = __fdiv_rn(num, den);
  inv.y = fmaf(-inv.x, den, num) * inv.x * (own ? 1.0f / kE4m3Max : 1.0f);
#pragma unroll 1
  for (int k0 = 0; k0 < TPW; k0 += kHold) {
    if (TPW > kHold) {
#pragma unroll
      for (int k = 0; k < kHold; ++k) {
        const int t = t_lo + k0 + k;
        if (have(t)) row[k].load(a, b, t - start, t, lane);
      }
    }
#pragma unroll
    for (int k = 0; k < kHold; ++k) {
      const int t = t_lo + k0 + k;
      if (have(t)) row[k].store_fp8(a, cache + (row0 + (t - base)) * kDqk, inv, lane);
    }
  }
  if (warp == w0 && lane == 0) a.scales[brow / G] = scale;
}

bool al(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

// Whether rows of kRopeDims at these three sizes and strides lie apart: taken by
// rising stride, each dim steps over all that the ones before it cover (any
// order of the dims, any slice).
bool apart(int n0, int64_t st0, int n1, int64_t st1, int n2, int64_t st2) {
  struct {
    int64_t n, step;
  } d[3] = {{n0, st0}, {n1, st1}, {n2, st2}};
  std::sort(d, d + 3, [](auto& x, auto& y) { return x.step < y.step; });
  int64_t cover = kRopeDims;
  for (auto& k : d) {
    if (k.n == 1) continue;
    if (k.step < cover || k.step > (INT64_MAX - cover) / (k.n - 1)) return false;
    cover += (k.n - 1) * k.step;
  }
  return true;
}

// Checks shared by the two entry points; fills everything but the pages.
int prepare_rope(RopeArgs* a, const void* kv_new, int64_t kv_sb, int64_t kv_ss, const void* q_rope,
                 int64_t q_sb, int64_t q_ss, int64_t q_sh, void* q_out, int64_t qo_sb,
                 int64_t qo_ss, int64_t qo_sh, void* cache, int num_pages,
                 const int32_t* block_table, int max_pages, const int32_t* seqlens,
                 const int32_t* new_lens, const float* cos_sin, int max_pos, int interleaved,
                 int batch, int s_new, int h_q) {
  if (!kv_new || !cache || !block_table || !seqlens || !cos_sin || batch < 1 || s_new < 1 ||
      num_pages < 1 || max_pages < 1 || max_pos < 1 || (q_rope == nullptr) != (q_out == nullptr) ||
      (int64_t)num_pages * kPageTokens >= ((int64_t)1 << 31) ||
      (int64_t)batch * s_new >= ((int64_t)1 << 31))
    return MLA_ERR_INVALID_ARG;
  if (!al(kv_new, 16) || !al(cache, 16) || !al(cos_sin, 16) || !al(block_table, 4) ||
      !al(seqlens, 4) || !al(new_lens, 4) || kv_sb < 0 || kv_ss < 0 || (kv_sb & 7) || (kv_ss & 7))
    return MLA_ERR_INVALID_ARG;
  if (q_rope) {
    if (h_q < 1 || !al(q_rope, 16) || !al(q_out, 16) ||
        ((q_sb | q_ss | q_sh | qo_sb | qo_ss | qo_sh) & 7) || q_sb < 0 || q_ss < 0 || q_sh < 0)
      return MLA_ERR_INVALID_ARG;
    // rows that are written must not lie on one another
    if (!apart(batch, qo_sb, s_new, qo_ss, h_q, qo_sh)) return MLA_ERR_INVALID_ARG;
  }
  a->kv_new = static_cast<const __nv_bfloat16*>(kv_new);
  a->kv_sb = kv_sb;
  a->kv_ss = kv_ss;
  a->q_in = static_cast<const __nv_bfloat16*>(q_rope);
  a->q_out = static_cast<__nv_bfloat16*>(q_out);
  a->qi_sb = q_sb;
  a->qi_ss = q_ss;
  a->qi_sh = q_sh;
  a->qo_sb = qo_sb;
  a->qo_ss = qo_ss;
  a->qo_sh = qo_sh;
  a->cache = cache;
  a->scales = nullptr;
  a->num_pages = num_pages;
  a->max_pages = max_pages;
  a->block_table = block_table;
  a->seqlens = seqlens;
  a->new_lens = new_lens;
  a->cos_sin = cos_sin;
  a->max_pos = max_pos;
  a->interleaved = interleaved ? 1 : 0;
  a->batch = batch;
  a->s_new = s_new;
  a->h_q = q_rope ? h_q : 0;
  return MLA_OK;
}

// The grid: `chunks` append CTAs for each entry, then the query CTAs.
int rope_grid(RopeArgs* a, int64_t chunks, int* grid) {
  int device = 0, sms = 0;
  const int st = device_current(&device, &sms, &a->err);
  if (st != MLA_OK) return st;
  a->chunks = (int)chunks;
  a->append_ctas = chunks * a->batch;
  const int64_t tokens = (int64_t)a->batch * a->s_new;
  // Four heads a thread where that still leaves every SM two CTAs (4096 tokens:
  // 29.2 us against 35.9 with one, bf16 pages, inputs not in L2; 16 tokens, which
  // take one: 4.4 us against 5.3 with four).
  const bool wide = tokens * ((a->h_q + 4 * kQHeads - 1) / (4 * kQHeads)) >= 2 * (int64_t)sms;
  a->heads_per_thread = wide ? 4 : 1;
  a->head_steps = (a->h_q + a->heads_per_thread * kQHeads - 1) / (a->heads_per_thread * kQHeads);
  const int64_t total = a->append_ctas + tokens * a->head_steps;
  if (total >= ((int64_t)1 << 31)) return MLA_ERR_INVALID_ARG;
  *grid = (int)total;
  return MLA_OK;
}

struct RopeLaunch {
  cudaLaunchConfig_t cfg;
  cudaLaunchAttribute attr[1];
  RopeLaunch(int grid, void* stream) {
    cfg = cudaLaunchConfig_t{};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(kRopeThreads);
    cfg.stream = static_cast<cudaStream_t>(stream);
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
  }
};

template <int HPT>
cudaError_t launch_rope_fp8(const cudaLaunchConfig_t& cfg, const RopeArgs& a, int tokens_per_warp,
                            int scale_tokens) {
  switch (tokens_per_warp) {
    case 1: return cudaLaunchKernelEx(&cfg, mla_rope_append_fp8_kernel<1, HPT>, a, scale_tokens);
    case 2: return cudaLaunchKernelEx(&cfg, mla_rope_append_fp8_kernel<2, HPT>, a, scale_tokens);
    case 4: return cudaLaunchKernelEx(&cfg, mla_rope_append_fp8_kernel<4, HPT>, a, scale_tokens);
    default: return cudaLaunchKernelEx(&cfg, mla_rope_append_fp8_kernel<8, HPT>, a, scale_tokens);
  }
}

}  // namespace
}  // namespace mla

using namespace mla;

extern "C" {

int mla_rope_append(const void* kv_new, int64_t kv_stride_b, int64_t kv_stride_s,
                    const void* q_rope, int64_t q_stride_b, int64_t q_stride_s, int64_t q_stride_h,
                    void* q_out, int64_t q_out_stride_b, int64_t q_out_stride_s,
                    int64_t q_out_stride_h, void* kv_cache, int num_pages,
                    const int32_t* block_table, int max_pages, const int32_t* cache_seqlens,
                    const int32_t* new_lens, const float* cos_sin, int max_positions,
                    int interleaved, int batch, int s_new, int h_q, void* stream) {
  RopeArgs a;
  int rc = prepare_rope(&a, kv_new, kv_stride_b, kv_stride_s, q_rope, q_stride_b, q_stride_s,
                        q_stride_h, q_out, q_out_stride_b, q_out_stride_s, q_out_stride_h, kv_cache,
                        num_pages, block_table, max_pages, cache_seqlens, new_lens, cos_sin,
                        max_positions, interleaved, batch, s_new, h_q);
  if (rc != MLA_OK) return rc;
  int grid = 0;
  rc = rope_grid(&a, ((int64_t)s_new + kRopeWarps - 1) / kRopeWarps, &grid);
  if (rc != MLA_OK) return rc;
  RopeLaunch l(grid, stream);
  const cudaError_t e = a.heads_per_thread == 4
                            ? cudaLaunchKernelEx(&l.cfg, mla_rope_append_kernel<4>, a)
                            : cudaLaunchKernelEx(&l.cfg, mla_rope_append_kernel<1>, a);
  return e == cudaSuccess ? MLA_OK : MLA_ERR_CUDA;
}

int mla_rope_append_fp8(const void* kv_new, int64_t kv_stride_b, int64_t kv_stride_s,
                        const void* q_rope, int64_t q_stride_b, int64_t q_stride_s,
                        int64_t q_stride_h, void* q_out, int64_t q_out_stride_b,
                        int64_t q_out_stride_s, int64_t q_out_stride_h, void* kv_cache,
                        float* scales, int scale_tokens, int num_pages, const int32_t* block_table,
                        int max_pages, const int32_t* cache_seqlens, const int32_t* new_lens,
                        const float* cos_sin, int max_positions, int interleaved, int batch,
                        int s_new, int h_q, void* stream) {
  if (!scales || !al(scales, 4) || scale_tokens < 1 || scale_tokens > kPageTokens ||
      (scale_tokens & (scale_tokens - 1)))
    return MLA_ERR_INVALID_ARG;
  RopeArgs a;
  int rc = prepare_rope(&a, kv_new, kv_stride_b, kv_stride_s, q_rope, q_stride_b, q_stride_s,
                        q_stride_h, q_out, q_out_stride_b, q_out_stride_s, q_out_stride_h, kv_cache,
                        num_pages, block_table, max_pages, cache_seqlens, new_lens, cos_sin,
                        max_positions, interleaved, batch, s_new, h_q);
  if (rc != MLA_OK) return rc;
  a.scales = scales;
  const int span = scale_tokens < kRopeWarps ? kRopeWarps : scale_tokens;
  int grid = 0;
  // s_new consecutive positions touch at most this many aligned spans
  rc = rope_grid(&a, ((int64_t)s_new + span - 2) / span + 1, &grid);
  if (rc != MLA_OK) return rc;
  RopeLaunch l(grid, stream);
  const cudaError_t e = a.heads_per_thread == 4
                            ? launch_rope_fp8<4>(l.cfg, a, span / kRopeWarps, scale_tokens)
                            : launch_rope_fp8<1>(l.cfg, a, span / kRopeWarps, scale_tokens);
  return e == cudaSuccess ? MLA_OK : MLA_ERR_CUDA;
}

}  // extern "C"
