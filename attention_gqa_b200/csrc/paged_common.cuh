// Device code that the attention kernels over a paged cache share: constants of the
// softmax, the search for a CTA's work, and the look-up of pages.
#pragma once

#include <atomic>
#include <cfloat>
#include <cmath>
#include <cstdint>

#include "internal.h"
#include "paged.h"
#include "sm100_ptx.cuh"

namespace gqa {
namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kScaleLog2 = 0.125f * kLog2e;
// The running maximum follows the scores only when one exceeds it by this much
// (log2 units): p then stays below 2^8, and most tiles leave the sums alone.
constexpr float kRescaleThreshold = 8.0f;
// A running maximum below every score: 2^(kNoMax - x) is 0 for any finite x.
constexpr float kNoMax = -FLT_MAX;

// Allows a kernel `bytes` of dynamic shared memory, once per device.
inline cudaError_t allow_shared(const void* kernel, uint32_t bytes, std::atomic<uint64_t>* prepared) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = uint64_t{1} << (dev & 63);
  if (prepared->load(std::memory_order_acquire) & bit) return cudaSuccess;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           static_cast<int>(bytes));
  if (e == cudaSuccess) prepared->fetch_or(bit, std::memory_order_release);
  return e;
}

struct ScanSlot {
  int row, split, chunks, part, len, unused;
};

// Length of sequence b, clamped to the table; one outside it is reported.
__device__ __forceinline__ int length_of(const PagedAttentionArgs& a, int b) {
  int len = __ldg(a.len + b);
  if (len < 0 || len > a.max_len) {
    atomicOr(a.err, kErrLength);
    len = len < 0 ? 0 : a.max_len;
  }
  return len;
}

// Sequence of a row.
__device__ __forceinline__ int sequence_of(const PagedAttentionArgs& a, int row) {
  return a.groups == 1 ? row : row / a.groups;
}

template <int NT, int kTile>
__device__ __forceinline__ int row_tiles(const PagedAttentionArgs& a, int row) {
  const int b = sequence_of(a, row);
  int lo, hi;
  paged_row_range(length_of(a, b), a.n, (row - b * a.groups) * NT, NT, a.window, &lo, &hi);
  return paged_row_tiles(lo, hi, kTile);
}

// Inclusive sums over the lanes.
__device__ __forceinline__ uint32_t warp_scan(uint32_t v, int lane) {
#pragma unroll
  for (int d = 1; d < 32; d *= 2) {
    const uint32_t u = __shfl_up_sync(0xffffffffu, v, d);
    if (lane >= d) v += u;
  }
  return v;
}

// The rows of one thread: their tiles and chunks. kRows consecutive ones at most. All rows
// are fewer than kPagedManyRows, so that their chunks, in the low half of a word, and the
// chunks of cut rows, in its high half, stay below 2^16.
template <int NT, int kTile, int kRows>
struct PlanRows {
  int r0, r1, tiles[kRows], n[kRows];
  __device__ __forceinline__ uint32_t load(const PagedAttentionArgs& a, int first, int last) {
    r0 = min(a.rows, first);
    r1 = min(a.rows, last);
    uint32_t sum = 0;
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      tiles[i] = r0 + i < r1 ? row_tiles<NT, kTile>(a, r0 + i) : 0;
      sum += static_cast<uint32_t>(tiles[i]);
    }
    return sum;
  }
  // into chunks of so many tiles; their counts
  __device__ __forceinline__ uint32_t cut(int chunk) {
    uint32_t sum = 0;
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      n[i] = r0 + i < r1 ? paged_row_chunks(tiles[i], chunk) : 0;
      sum += words(i);
    }
    return sum;
  }
  // looks for chunk `cid` here, before whose rows lie the counts `at`
  __device__ __forceinline__ void find(const PagedAttentionArgs& a, int cid, uint32_t at,
                                       ScanSlot* slot) const {
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      const int split = cid - static_cast<int>(at & 0xFFFFu);
      if (split >= 0 && split < n[i]) {
        slot->row = r0 + i;
        slot->split = split;
        slot->chunks = n[i];
        slot->part = static_cast<int>(at >> 16);
        slot->len = min(max(__ldg(a.len + sequence_of(a, r0 + i)), 0), a.max_len);
      }
      at += words(i);
    }
  }
  __device__ __forceinline__ uint32_t words(int i) const {
    return static_cast<uint32_t>(n[i]) * (n[i] > 1 ? 0x10001u : 1u);
  }
};

// Finds chunk `cid` of the call, by all kThreads threads of the CTA; false past the
// last one. `sums`: two words per warp.
//
// Every CTA begins with this, so it is kept short: where no row is cut, chunks are rows (which
// saves a window of 128 over 64 sequences 0.9 of 9 us, and 1024 ragged sequences of up to
// 1024 bf16 take 186 us); up to 96 rows the first warp does it alone; more, below 1024, are
// spread over all threads (1023 of those: 210 us). Those need no estimate of whether whole rows end
// first: with 97 rows of many tokens and 55 chunks aimed for, only rows of more than 1.7
// times the average are cut at all.
template <int NT, int kTile, int kThreads>
__device__ __forceinline__ bool find_chunk(const PagedAttentionArgs& a, int cid, uint32_t* sums,
                                           ScanSlot* slot) {
  constexpr int kWarps = kThreads / 32;
  const int t = static_cast<int>(threadIdx.x);
  const int warp = t >> 5, lane = t & 31;
  if (a.none_cut) {
    if (t == 0) {
      slot->row = cid;
      slot->split = slot->part = 0;
      slot->chunks = 1;
      slot->len = length_of(a, sequence_of(a, cid));
    }
    __syncthreads();
    return true;  // the grid has no more
  }
  if (t == 0) slot->row = -1;
  constexpr int kFew = 3;
  if (a.rows <= 32 * kFew) {
    if (warp == 0) {
      const int per = (a.rows + 31) / 32;
      PlanRows<NT, kTile, kFew> rows;
      const uint32_t total =
          __reduce_add_sync(0xffffffffu, rows.load(a, lane * per, lane * per + per));
      int chunk = paged_chunk_tiles(total, a.target);
      uint32_t mine = rows.cut(chunk);
      if (a.one_wave || NT > 2) {
        int count = static_cast<int>(__reduce_add_sync(0xffffffffu, mine & 0xFFFFu));
        // (ends: chunks grow until every row is one, and the rows are fewer than a wave)
        while (a.one_wave && count > a.wave) {
          chunk = paged_longer_chunk(chunk, count, a.wave);
          mine = rows.cut(chunk);
          count = static_cast<int>(__reduce_add_sync(0xffffffffu, mine & 0xFFFFu));
        }
        if (!a.one_wave) {
          int longest = 0, whole = 0;
#pragma unroll
          for (int i = 0; i < kFew; ++i) {
            if (rows.n[i] > 0) longest = max(longest, (rows.tiles[i] + rows.n[i] - 1) / rows.n[i]);
            whole = max(whole, rows.tiles[i]);
          }
          longest = __reduce_max_sync(0xffffffffu, longest);
          whole = __reduce_max_sync(0xffffffffu, whole);
          if (paged_estimate(total, a.rows, whole, a.wave, false) <=
              paged_estimate(total, count, longest, a.wave, true))
            mine = rows.cut(whole);
        }
      }
      rows.find(a, cid, warp_scan(mine, lane) - mine, slot);
    }
  } else {
    const int per = (a.rows + kThreads - 1) / kThreads;
    PlanRows<NT, kTile, (kPagedManyRows - 1 + kThreads - 1) / kThreads> rows;
    const uint32_t part = __reduce_add_sync(0xffffffffu, rows.load(a, t * per, t * per + per));
    if (lane == 0) sums[warp] = part;
    __syncthreads();
    uint32_t total = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) total += sums[w];
    const uint32_t mine = rows.cut(paged_chunk_tiles(total, a.target));
    const uint32_t inc = warp_scan(mine, lane);
    if (lane == 31) sums[kWarps + warp] = inc;
    __syncthreads();
    uint32_t at = inc - mine;
#pragma unroll
    for (int w = 0; w < kWarps - 1; ++w)
      if (w < warp) at += sums[kWarps + w];
    rows.find(a, cid, at, slot);
  }
  __syncthreads();
  return slot->row >= 0;
}

// Four e4m3 codes to two f16x2 words (exact).
__device__ __forceinline__ void e4m3x4_to_f16(uint32_t codes, uint32_t& lo, uint32_t& hi) {
  asm("{\n\t.reg .b16 l, u;\n\tmov.b32 {l, u}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, l;\n\t"
      "cvt.rn.f16x2.e4m3x2 %1, u;\n\t}"
      : "=r"(lo), "=r"(hi)
      : "r"(codes));
}

// Four e4m3 codes to their values.
__device__ __forceinline__ void e4m3x4_to_f32(uint32_t codes, float (&x)[4]) {
  uint32_t lo, hi;
  e4m3x4_to_f16(codes, lo, hi);
  asm("{\n\t.reg .b16 l, u;\n\tmov.b32 {l, u}, %2;\n\tcvt.f32.f16 %0, l;\n\tcvt.f32.f16 %1, u;\n\t}"
      : "=f"(x[0]), "=f"(x[1])
      : "r"(lo));
  asm("{\n\t.reg .b16 l, u;\n\tmov.b32 {l, u}, %2;\n\tcvt.f32.f16 %0, l;\n\tcvt.f32.f16 %1, u;\n\t}"
      : "=f"(x[2]), "=f"(x[3])
      : "r"(hi));
}

struct PageEntry {
  int page;
  float ks, vs;
};

// Page `pi` of a sequence and its scales for kv head g. Pages before the one of the
// first visible key `lo`, or past the last, are not looked at (their entries may be
// unset); a bad number is reported, and stands for a page past the pool, of which
// copies read zeros. Both have a value scale below 0.
template <bool kFp8>
__device__ __forceinline__ PageEntry fetch_page(const PagedAttentionArgs& a, const int32_t* table,
                                                int pi, int lo, int last_page, int g) {
  PageEntry e = {a.cache.num_pages, 1.f, -1.f};
  if (pi <= last_page && pi >= (lo >> a.cache.page_log2)) {
    const int page = __ldg(table + pi);
    if (paged_page_ok(page, a.cache.num_pages)) {
      e.page = page;
      if (kFp8) {
        e.ks = __ldg(a.cache.k_scale + static_cast<int64_t>(page) * kNumKvHeads + g);
        e.vs = __ldg(a.cache.v_scale + static_cast<int64_t>(page) * kNumKvHeads + g);
      }
    } else {
      atomicOr(a.err, kErrPage);
    }
  }
  return e;
}

// What the softmax needs of a page's scales: the factor of its scores, log2 of its value
// scale in the chunk's unit (paged.h), and that scale's reciprocal. Sets *far if the scale
// lies too far from the unit.
__device__ __forceinline__ float4 page_factors(float ks, float vs, int unit, volatile int* far) {
  // (zeros have the least scale, so that they do not raise the maximum above the others)
  const float v = vs < 0.f ? kScaleNear : vs * paged_power(-unit);
  if (paged_scale_far(v)) *far = 1;  // (what the factors make of it is not used)
  return make_float4(ks * kScaleLog2, log2f(v), 1.f / v, 0.f);
}

// Normalises a chunk's sums for the joining kernel where values are in a unit: the row's M and
// sum become those of the same weights with a sum in [1/4, 1/2), and its elements are to be
// multiplied by both factors returned, one after the other. They are then no
// larger than the output, and overflow only where that does.
__device__ __forceinline__ float2 to_part(float* M, float* sum, int unit) {
  if (!(*M > kNoMax)) return make_float2(1.f, 1.f);
  const int k = min(max(static_cast<int>(__float_as_uint(*sum) >> 23) - 127 + 2, -126), 126);
  *M += static_cast<float>(k);
  *sum *= paged_power(-k);
  return make_float2(paged_power(-k), paged_power(unit));
}

// The formula itself, for a chunk with value scales too far apart (e4m3 pages): a half-warp
// takes one head of one token over the keys [key_a, key_b) that the token sees, lane e of it
// elements 4e .. 4e+3, and writes the output (the row's only chunk) or its part. Sums are in
// 64 bits, which hold every product of a weight, a scale and a code. One key after the other,
// and as slow as such scales are rare (64 sequences of 8192, every chunk with them: 5.9 ms
// against 0.1). Both half-warps of a warp come with the same token.
__device__ __forceinline__ void plain_row(const PagedAttentionArgs& a, int b, int t, int idx,
                                          int head, int key_a, int key_b, int chunks,
                                          int64_t part_row) {
  const int lane = static_cast<int>(threadIdx.x & 31);
  const int g = head / kGroup, d0 = (lane & 15) * 4, page_log2 = a.cache.page_log2;
  float y[4] = {0.f, 0.f, 0.f, 0.f};
  if (idx >= 0) {
    int p = a.pos ? __ldg(a.pos + static_cast<int64_t>(b) * a.n + t) : idx;
    p = min(max(p, 0), kMaxPosition - 1);  // (reported by the others)
    const uint16_t* q = a.q + b * a.q_batch + t * a.q_token + head * kHeadDim;
    const float2* row = a.rope + static_cast<int64_t>(p) * kRopePairs + (d0 & 31);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float2 f = __ldg(row + e);
      const float x = bf16lo_to_f32(__ldg(q + d0 + e)), z = bf16lo_to_f32(__ldg(q + (d0 ^ 32) + e));
      y[e] = fmaf(x, f.x, (d0 < 32 ? -z : z) * f.y);
    }
  }
  const int32_t* table = a.table + static_cast<int64_t>(b) * a.max_pages;
  const int first = a.window > 0 ? max(idx - a.window + 1, key_a) : key_a;
  const int last = min(idx + 1, key_b);
  float m = kNoMax;
  double l = 0., o[4] = {0., 0., 0., 0.};
#pragma unroll 1
  for (int key = first; key < last; ++key) {
    const int page = __ldg(table + (key >> page_log2));
    uint32_t kc = 0, vc = 0;  // a bad page's
    float ks = 1.f, vs = 1.f;
    if (paged_page_ok(page, a.cache.num_pages)) {
      const int64_t at = page * a.cache.page_stride +
                         (key & ((1 << page_log2) - 1)) * a.cache.token_stride +
                         g * a.cache.head_stride + d0;
      kc = *reinterpret_cast<const uint32_t*>(a.cache.k + at);
      vc = *reinterpret_cast<const uint32_t*>(a.cache.v + at);
      ks = __ldg(a.cache.k_scale + static_cast<int64_t>(page) * kNumKvHeads + g);
      vs = __ldg(a.cache.v_scale + static_cast<int64_t>(page) * kNumKvHeads + g);
    }
    float k[4], v[4];
    e4m3x4_to_f32(kc, k);
    e4m3x4_to_f32(vc, v);
    float x = fmaf(y[0], k[0], fmaf(y[1], k[1], fmaf(y[2], k[2], y[3] * k[3])));
#pragma unroll
    for (int w = 8; w > 0; w /= 2) x += __shfl_xor_sync(0xffffffffu, x, w);
    x *= ks * kScaleLog2;
    if (x > m) {
      const double f = ex2_approx(m - x);
      m = x;
      l *= f;
#pragma unroll
      for (int e = 0; e < 4; ++e) o[e] *= f;
    }
    const double p = ex2_approx(x - m);
    l += p;
#pragma unroll
    for (int e = 0; e < 4; ++e) o[e] += p * (static_cast<double>(vs) * v[e]);
  }
  if (chunks == 1) {
    const float sink = __ldg(a.sinks + head) * kLog2e;
    const float top = fmaxf(sink, m);
    const double f = ex2_approx(m - top);
    const double scale = m > kNoMax ? f / (f * l + ex2_approx(sink - top)) : 0.;
    *reinterpret_cast<uint2*>(
        a.out + ((static_cast<int64_t>(b) * a.n + t) * kNumHeads + head) * kHeadDim + d0) =
        make_uint2(pack_bf16x2(static_cast<float>(o[0] * scale), static_cast<float>(o[1] * scale)),
                   pack_bf16x2(static_cast<float>(o[2] * scale), static_cast<float>(o[3] * scale)));
  } else {
    // as to_part() leaves it
    const double unit = l > 0. ? 0.25 / l : 1.;
    *reinterpret_cast<float4*>(a.part_o + part_row * kHeadDim + d0) =
        make_float4(static_cast<float>(o[0] * unit), static_cast<float>(o[1] * unit),
                    static_cast<float>(o[2] * unit), static_cast<float>(o[3] * unit));
    if (d0 == 0)
      a.part_ml[part_row] =
          m > kNoMax ? make_float2(m + static_cast<float>(log2(4. * l)), 0.25f) : make_float2(m, 0.f);
  }
}

// Splits x and y into two bf16 terms each: returns the first ones, packed, and leaves the
// second ones, which the caller rounds. Terms of a value have its sign and neither is 0 unless
// it is: what multiplies them may be infinite, and 0 or terms of two signs would make that
// NaN. So the first term is cut off, not rounded (together 2^-16 of the value, where a rounded
// first one leaves 2^-17), and a value of one term gets a second one far below fp32's step.
__device__ __forceinline__ uint32_t split_bf16x2(float& x, float& y) {
  const uint32_t hi = __byte_perm(__float_as_uint(x), __float_as_uint(y), 0x7632);
  const float a = bf16lo_to_f32(hi), b = bf16hi_to_f32(hi);
  x = a == x ? x * 0x1p-25f : x - a;
  y = b == y ? y * 0x1p-25f : y - b;
  return hi;
}

__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

__device__ __forceinline__ uint4 lds128(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(addr));
  return v;
}

__device__ __forceinline__ void sts128(uint32_t addr, uint4 v) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(v.x), "r"(v.y),
               "r"(v.z), "r"(v.w)
               : "memory");
}

}  // namespace
}  // namespace gqa
