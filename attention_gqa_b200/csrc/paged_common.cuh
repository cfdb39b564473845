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
// Every CTA begins with this, so it is kept short: where no row is cut, chunks are rows (a
// window of 128 over 64 sequences takes 7.2 us, not 8.1, and 1024 ragged sequences of up to
// 1024 bf16 176 us); up to 96 rows the first warp does it alone; more, below 1024, are spread
// over all threads (1023 of those: 192 us).
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

struct PageEntry {
  int page;
  float ks, vs;
};

// Page `pi` of a sequence and its scales for kv head g. Pages before the one of the
// first visible key `lo`, or past the last, are not looked at (their entries may be
// unset); a bad number is reported, and stands for a page past the pool, of which
// copies read zeros.
template <bool kFp8>
__device__ __forceinline__ PageEntry fetch_page(const PagedAttentionArgs& a, const int32_t* table,
                                                int pi, int lo, int last_page, int g) {
  PageEntry e = {a.cache.num_pages, 1.f, 1.f};
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

// What the softmax needs of a page's scales: the factor of its scores, log2 of its
// value scale, and that scale's reciprocal.
__device__ __forceinline__ float4 page_factors(float ks, float vs) {
  vs = fmaxf(vs, 0x1p-100f);
  return make_float4(ks * kScaleLog2, log2f(vs), 1.f / vs, 0.f);
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

// Four e4m3 codes to two f16x2 words (exact).
__device__ __forceinline__ void e4m3x4_to_f16(uint32_t codes, uint32_t& lo, uint32_t& hi) {
  asm("{\n\t.reg .b16 l, u;\n\tmov.b32 {l, u}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, l;\n\t"
      "cvt.rn.f16x2.e4m3x2 %1, u;\n\t}"
      : "=r"(lo), "=r"(hi)
      : "r"(codes));
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
