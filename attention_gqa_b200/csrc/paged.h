// The paged key/value cache: what its host entry points and kernels agree on.
//
// The arithmetic here (which keys a row of queries sees, how the work is cut
// into chunks, where a token lies, which scale a page gets) is plain C++ that
// also compiles without CUDA, so it is tested on the CPU.
#pragma once

#include <cstddef>
#include <cstdint>
#include <cstring>

#ifdef __CUDACC__
#define GQA_HD __host__ __device__ __forceinline__
#else
#define GQA_HD inline
#endif

namespace gqa {

constexpr int kPagedTile = 64;   // keys per tile of the attention kernel for few tokens
constexpr int kPagedTileN = 128;  // and of the one for many

// Keys [lo, hi) that some token of one row of queries sees. A row is up to
// `nt` tokens of one sequence, the tokens t0 .. of the n newest; token t sits at
// index len - n + t (a negative index is no token and sees nothing).
GQA_HD void paged_row_range(int len, int n, int t0, int nt, int window, int* lo, int* hi) {
  const int last = t0 + nt < n ? t0 + nt : n;
  const int first_idx = len - n + t0;
  *hi = len - n + last > 0 ? len - n + last : 0;
  *lo = window > 0 && first_idx - window + 1 > 0 ? first_idx - window + 1 : 0;
}

GQA_HD int paged_row_tiles(int lo, int hi, int tile) {
  return hi > lo ? (hi - 1) / tile - lo / tile + 1 : 0;
}

// Rows of at most this many tiles are one chunk: a chunk's own latency is that
// of many tiles, and a row that is not cut needs no second kernel.
constexpr int kPagedWhole = 8;
// Calls of so many rows cut none: their CTAs fill the GPU many times over, and each would
// have to look at all the lengths to find its chunk. That is right for rows of like lengths
// (1024 ragged ones of up to 1024 bf16: 186 us, 1023 that are planned: 210), and costs most where
// one is far longer than all the others: of 131072 keys among 1023 of 64, bf16, it takes
// 0.99 ms for one token of each, where one row less takes 0.19 (e4m3 0.71 and 0.16; five
// tokens 1.8 and 0.43).
constexpr int kPagedManyRows = 1024;

// Whether no row is cut, of rows with at most `most` tiles.
GQA_HD bool paged_none_cut(int64_t rows, int most) {
  return most <= kPagedWhole || rows >= kPagedManyRows;
}

// No chunk of a longer row has fewer tiles than this, unless the division of its
// tiles into equal parts leaves one less.
constexpr int kPagedLeast = 4;

// Tiles per chunk when all rows together have `total` tiles and about `target`
// chunks are wanted.
GQA_HD int paged_chunk_tiles(int64_t total, int target) {
  const int64_t c = (total + target - 1) / target;
  return c < kPagedLeast ? kPagedLeast : static_cast<int>(c);
}

// A longer chunk to try when chunks of `chunk` tiles came to `count`, more than `wave`.
GQA_HD int paged_longer_chunk(int chunk, int count, int wave) {
  return static_cast<int>((static_cast<int64_t>(chunk) * count + wave - 1) / wave);
}

// Estimated time, in `wave`-ths of a tile's, of `count` chunks of at most `longest` and
// together `total` tiles on `wave` places, for the kernel for many tokens: a chunk costs
// three tiles before its first, and joining cut rows two in all. Equal chunks run in whole
// waves, unequal ones are dealt out as places get free.
GQA_HD int64_t paged_estimate(int64_t total, int count, int longest, int wave, bool cut) {
  const int64_t one = longest + 3;
  int64_t t = (count + wave - 1) / wave * wave * one;
  if (count > wave) {
    const int64_t dealt = total + 3 * static_cast<int64_t>(count) + wave * one / 2;
    t = dealt < t ? dealt : t;
  }
  return t + (cut ? 2 * wave : 0);
}

// Chunks of one row (a row without keys has one too: it writes the zeros).
GQA_HD int paged_row_chunks(int tiles, int chunk) {
  return tiles > chunk && tiles > kPagedWhole ? (tiles + chunk - 1) / chunk : 1;
}

// Chunks of a whole call are at most this many, when no row has more than `most`
// tiles: sum of max(1, ceil(tiles/c)), with c >= total/target and c >= kPagedLeast.
GQA_HD int64_t paged_max_chunks(int64_t rows, int most, int target) {
  if (paged_none_cut(rows, most)) return rows;
  const int64_t cut = rows * most / kPagedLeast;
  return rows + (cut < target ? cut : target);
}

// Chunks of rows that have more than one: those leave partial sums in the
// workspace. Such a row has more than c tiles, so ceil(tiles/c) < 2 tiles/c.
GQA_HD int64_t paged_max_parts(int target) { return 2 * static_cast<int64_t>(target); }

// Chunks aimed for beyond one wave, by the tokens of a row (for 148 SMs; the workspace is
// made for so many).
GQA_HD int paged_target(int row_tokens) { return row_tokens <= 2 ? 111 : 55; }

// Chunks that a GPU of so many SMs holds at a time: eight CTAs of the kernel for few tokens,
// one per kv head, are a chunk, four of the other. No more than the workspace has parts for.
GQA_HD int paged_wave(int row_tokens, int num_sms) {
  const int per_sm = row_tokens == 1 ? 4 : row_tokens == 2 ? 3 : 2;
  const int parts = static_cast<int>(paged_max_parts(paged_target(row_tokens)));
  const int wave = num_sms * per_sm / 8;
  return wave < 1 ? 1 : wave < parts ? wave : parts;
}

// Tiles [*a, *b) of a row's `tiles` that chunk `i` of `chunks` takes.
GQA_HD void paged_chunk_range(int tiles, int chunks, int i, int* a, int* b) {
  *a = static_cast<int>(static_cast<int64_t>(tiles) * i / chunks);
  *b = static_cast<int>(static_cast<int64_t>(tiles) * (i + 1) / chunks);
}

GQA_HD bool paged_page_ok(int page, int num_pages) { return page >= 0 && page < num_pages; }

// Whether an append of `count` of at most `n` tokens that ends at `len` stays
// inside a sequence of max_len tokens.
GQA_HD bool paged_append_ok(int len, int count, int n, int max_len) {
  return count >= 0 && count <= n && len >= count && len <= max_len;
}

// Exponents a page's scale may have: 448 * 2^120 holds every finite bf16, and
// values below 2^-64 need no finer steps.
constexpr int kScaleLow = -64;
constexpr int kScaleHigh = 120;

// Bits of the least power of two 2^e with `largest` <= 448 * 2^e, e limited to
// [kScaleLow, kScaleHigh]; `largest_bits` are those of a finite fp32 >= 0.
// 448 = 1.75 * 2^8: a value m * 2^x (1 <= m < 2) needs e = x - 8, or x - 7 above 1.75.
GQA_HD uint32_t paged_scale_bits(uint32_t largest_bits) {
  int e = static_cast<int>(largest_bits >> 23) - 127 - 8;
  if ((largest_bits & 0x7FFFFFu) > 0x600000u) ++e;
  if (e < kScaleLow) e = kScaleLow;
  if (e > kScaleHigh) e = kScaleHigh;
  return static_cast<uint32_t>(e + 127) << 23;
}

// 2^e as fp32, -126 <= e <= 127.
GQA_HD float paged_power(int e) {
  const uint32_t bits = static_cast<uint32_t>(e + 127) << 23;
  float x;
  memcpy(&x, &bits, sizeof x);
  return x;
}

// The unit (a power of two) that a chunk's values are summed in: about the first page's
// scale. Weights are multiplied by a page's value scale s before they are rounded and
// summed, w = 2^(x - M) s, and the normaliser takes w / s back. That needs 2^(x - M) s to
// stay inside fp32's exponents for every x that counts, down to 2^-30 of the largest weight:
// scales between 2^-76 and 2^20 of the unit leave it above 2^-126. Not below 2^-16, as
// a first page of zeros has a scale of 2^-64, and says nothing of the others.
constexpr int kUnitLow = -16, kUnitHigh = 126;
GQA_HD int paged_unit(float scale) {  // below 0: no scale
  if (!(scale >= 0.f)) return 0;
  uint32_t bits;
  memcpy(&bits, &scale, sizeof bits);
  const int e = static_cast<int>(bits >> 23) - 127;
  return e < kUnitLow ? kUnitLow : e > kUnitHigh ? kUnitHigh : e;
}

// Whether a scale in that unit lies outside.
constexpr float kScaleNear = 0x1p-76f;
GQA_HD bool paged_scale_far(float scale) { return !(scale >= kScaleNear && scale <= 0x1p20f); }

// Whether a value (bits of a finite fp32 >= 0) lies within 16 ulps of where its scale
// changes, 1.75 * 2^x.
GQA_HD bool paged_near_border(uint32_t bits) {
  return (bits & 0x7FFFFFu) - (0x600000u - 16u) <= 32u;
}

}  // namespace gqa
