// Attention of the newest tokens of each sequence over a paged key/value cache,
// for sm_100a: grouped queries, sliding window and per-head sink as in the other
// entry points; pages of bf16, or of e4m3 with a scale per page and kv head.
//
// Work. A row is up to NT consecutive query tokens of one sequence. Its visible
// keys are cut into tiles of 64, and all rows' tiles into chunks of about equal
// length (paged.h): every CTA finds its (row, chunk, kv head) by a scan over the
// lengths, so the work follows the lengths on the device and not the capacity of
// the table. Chunks of a row that has several leave partial sums, which the
// combine kernel joins; a row's only chunk writes its output itself.
//
// Orientation. Products run transposed, keys (or head_dim) in the 16 rows of
// mma.m16n8k16 and the 8 query heads of a group in its 8 columns:
//   S^T = K Q^T, O^T = V^T P^T,
// so one token wastes no half of an instruction, and K and V fragments serve all
// NT tokens. Each of four warps takes 16 keys of every tile, with its own running
// maximum; the warps join at the end.
//
// Precision. bf16 pages: q and p are split into two bf16 terms (the second product
// costs tensor time that HBM leaves unused), which hold 16 bits; beside them only the sums'
// fp32 and the output round. e4m3 pages: codes are exact in f16, q is scaled by a power of two per head
// and rounded to f16 (2^-12), and so is p. A page's value scale s_v joins the
// exponent, w = 2^(x + log2 s_v - M), which keeps the largest w in f16's range whatever
// the scales are; the normaliser takes w / s_v in fp32. Scales are taken in a chunk's unit (paged.h),
// and a chunk whose scales are too far apart for that is done again by the formula itself.
//
// Bound by HBM where there is much to read, at 256 (bf16) or 128 (e4m3) bytes per key and
// head: 64 sequences of 8192 in bf16 pages take 166 us, 6.5 TB/s. e4m3 pages need as many
// instructions for half the bytes (the conversion of codes has half the rate of other
// arithmetic), and their warps wait on one another's results: 64 ragged sequences up to
// 8192 62 us, 4.5 TB/s; one of 131072 34 us, 4.0 TB/s. Short calls are the latency of the
// lengths, page numbers, tensor maps and pages in turn: one sequence of 257 keys 5.9 us.
//
// Two tokens at most: with four per row (mma.m16n8k16 for each) five drafted tokens of 16
// sequences took 142 us and a piece of 512 on 4096 718 us, against 49 and 103 of the
// first form of the kernel for many tokens, which in turn takes 125 to 245 us for two
// tokens of 8 x 32768 and 64 x 8192 where this one takes 86 and 157 (e4m3).
#include <cfloat>
#include <cmath>

#include "paged_common.cuh"

namespace gqa {
namespace {

constexpr int kWarps = 4;  // consumer warps
constexpr int kThreads = (kWarps + 1) * 32;
// Three stages leave shared memory for four CTAs of an SM (bf16, with four stages and three
// CTAs: 64 sequences of a window of 128 12.2 us against 8.1, as they are no longer one wave;
// the others alike).
constexpr int kStages = 3;
// Sixteen-key blocks a warp takes of a tile: two for e4m3, whose work per byte is
// twice as much, so that the waits and indices of a tile serve 32 keys (full sequences, 64 of
// 8192, 106 us against 122 with one block and five CTAs; bf16 reads at HBM's rate with one).
template <bool kFp8>
struct Shape {
  static constexpr int kElem = kFp8 ? 1 : 2;
  static constexpr int kBlocks = kFp8 ? 2 : 1;
  static constexpr int kTile = 16 * kWarps * kBlocks;  // keys
  static constexpr uint32_t kTileBytes = kTile * kHeadDim * kElem;  // one of K or V
};

template <bool kFp8, int NT>
struct Smem {
  static constexpr uint32_t kK = 0;
  static constexpr uint32_t kV = kK + kStages * Shape<kFp8>::kTileBytes;
  static constexpr uint32_t kTiles = kV + kStages * Shape<kFp8>::kTileBytes;
  // the warps' sums are joined where the tiles were
  static constexpr uint32_t kMergeWarp = NT * kGroup * (kHeadDim + 2) * 4;
  static constexpr uint32_t kMerge = 0;
  static constexpr uint32_t kEnd0 = kTiles > kWarps * kMergeWarp ? kTiles : kWarps * kMergeWarp;
  static constexpr uint32_t kQ = kEnd0;  // 16-bit [2][NT][8][64] (the second half: bf16 only)
  static constexpr uint32_t kQExp = kQ + (kFp8 ? 1 : 2) * NT * kGroup * kHeadDim * 2;  // [NT][8]
  // float4 [stages][blocks of a tile], e4m3
  static constexpr int kPages = kFp8 ? kWarps * Shape<kFp8>::kBlocks : 0;
  static constexpr uint32_t kPage = kQExp + NT * kGroup * 4;
  static constexpr uint32_t kBar = kPage + kStages * kPages * 16;
  static constexpr uint32_t kScan = kBar + 2 * kStages * 8;  // 5 + 5 warp sums, slot
  static constexpr uint32_t kMisc = kScan + 2 * 5 * 4 + sizeof(ScanSlot);
  static constexpr uint32_t kBytes = kMisc + 16 + 1024;
};

__device__ __forceinline__ void mma_bf16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                         uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ void mma_f16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                        uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Transposes an 8x8 matrix of 16-bit elements held one row pair per lane.
__device__ __forceinline__ uint32_t transpose8(uint32_t a) {
  uint32_t d;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
  return d;
}

template <bool kFp8, int NT>
__global__ void __launch_bounds__(kThreads, NT == 2 ? 3 : 4)
    paged_attention_kernel(const __grid_constant__ PagedMaps maps, const PagedAttentionArgs a) {
  using L = Smem<kFp8, NT>;
  constexpr int kTile = Shape<kFp8>::kTile;
  constexpr int kBlocks = Shape<kFp8>::kBlocks;
  constexpr uint32_t kTileBytes = Shape<kFp8>::kTileBytes;
  constexpr uint32_t kRowBytes = kHeadDim * Shape<kFp8>::kElem;
  griddep_launch_dependents();
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  const uint32_t sbase = smem_u32(smem);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + L::kMisc);
  volatile int* far = abort_flag + 1;   // e4m3: whether a value scale lies too far from
  volatile int* unit = abort_flag + 2;  // the chunk's unit
  auto full_bar = [&](int s) { return sbase + L::kBar + 8u * s; };
  auto empty_bar = [&](int s) { return sbase + L::kBar + 8u * (kStages + s); };
  const int warp = static_cast<int>(threadIdx.x >> 5);
  const int lane = static_cast<int>(threadIdx.x & 31);
  const int g = static_cast<int>(blockIdx.x % kNumKvHeads);

  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(full_bar(s), 1);
      mbar_init(empty_bar(s), kWarps);
    }
    fence_barrier_init();
  }
  if (threadIdx.x == 32 * kWarps) {
    prefetch_tensormap(&maps.k);
    prefetch_tensormap(&maps.v);
  }
  // The tokens, lengths and pages, and the workspace, may still be in use by
  // the kernel before.
  griddep_wait();
  if (threadIdx.x == 0) {
    *abort_flag = (*reinterpret_cast<volatile int*>(a.err) & kErrTimeout) ? 1 : 0;
    *far = *unit = 0;
  }
  ScanSlot* slot = reinterpret_cast<ScanSlot*>(smem + L::kScan + 2 * 5 * 4);
  if (!find_chunk<NT, kTile, kThreads>(a, static_cast<int>(blockIdx.x / kNumKvHeads),
                                       reinterpret_cast<uint32_t*>(smem + L::kScan), slot))
    return;  // past the call's last chunk
  const bool skip = *abort_flag != 0;
  const int row = slot->row, chunks = slot->chunks, part = slot->part + slot->split;
  if (a.meta && slot->split == 0 && g == 0 && threadIdx.x == 0)
    a.meta[row] = make_int2(slot->part, chunks);
  const int b = sequence_of(a, row);
  const int t0 = (row - b * a.groups) * NT;
  const int len = slot->len;
  const int idx0 = len - a.n + t0;  // index of the row's first token
  int lo, hi, tile_a, tile_b;
  paged_row_range(len, a.n, t0, NT, a.window, &lo, &hi);
  paged_chunk_range(paged_row_tiles(lo, hi, kTile), chunks, slot->split, &tile_a, &tile_b);
  const int key_a = (lo / kTile + tile_a) * kTile;  // first key of the chunk's tiles
  const int n_tiles = tile_b - tile_a;
  const int page_log2 = a.cache.page_log2;

  if (warp == kWarps) {
    // ---------------------------------------------------------------- producer
    if (!skip && n_tiles > 0) {
      const int P = 1 << page_log2;
      const int box = P < kPagedTile ? P : kPagedTile;  // keys per copy
      const int boxes = kTile / box;                    // at most 8
      const int last_page = (hi - 1) >> page_log2;
      const int32_t* table = a.table + static_cast<int64_t>(b) * a.max_pages;
      // Lane i holds page number pbase + i of the sequence, and its scales; the next
      // 32 are loaded while these are used.
      auto fetch = [&](int pi) { return fetch_page<kFp8>(a, table, pi, lo, last_page, g); };
      int pbase = key_a >> page_log2;
      PageEntry cur = fetch(pbase + lane), nxt = fetch(pbase + 32 + lane);
      int in = 0;  // the chunk's unit
      if (kFp8) {
        in = paged_unit(__shfl_sync(0xffffffffu, cur.vs, (max(key_a, lo) >> page_log2) - pbase));
        if (lane == 0) *unit = in;
      }
      const int sub = lane & 7;
      int issued = 0;
      int s = 0;             // stage of tile i
      uint32_t phase = 1;    // parity of its release before; a fresh barrier passes at once
      for (int i = 0; i < n_tiles; ++i) {
        const int key0 = key_a + i * kTile;
        if ((key0 >> page_log2) >= pbase + 32) {
          pbase += 32;
          cur = nxt;
          nxt = fetch(pbase + 32 + lane);
        }
        if (!mbar_wait_warp(empty_bar(s), phase, abort_flag, a.err, kErrTimeout, kWaitTimeoutNs))
          break;
        // pages of this tile that hold a visible key
        const int key = key0 + sub * box;
        const int page = __shfl_sync(0xffffffffu, cur.page, ((key >> page_log2) - pbase) & 31);
        const bool load = sub < boxes && key < hi && key + box > lo;
        const int n_load = __popc(__ballot_sync(0xffffffffu, load) & 0xFFu);
        if (lane == 0)
          mbar_expect_tx(full_bar(s), 2u * static_cast<uint32_t>(n_load * box) * kRowBytes);
        __syncwarp();
        if (load && lane < 16) {
          const uint32_t dst = sbase + (lane < 8 ? L::kK : L::kV) + s * kTileBytes +
                               static_cast<uint32_t>(sub * box) * kRowBytes;
          tma_load_4d(dst, lane < 8 ? &maps.k : &maps.v, full_bar(s), 0, g, key & (P - 1), page);
        }
        if (kFp8) {
          const int pw = (key0 + sub * 16) >> page_log2;  // page of a block of 16 keys
          const float ks = __shfl_sync(0xffffffffu, cur.ks, (pw - pbase) & 31);
          const float vs = __shfl_sync(0xffffffffu, cur.vs, (pw - pbase) & 31);
          if (lane < L::kPages)
            *reinterpret_cast<float4*>(smem + L::kPage + (s * L::kPages + lane) * 16) =
                page_factors(ks, vs, in, far);
          __syncwarp();
        }
        if (lane == 0) mbar_arrive(full_bar(s));  // and the scales are there
        if (++s == kStages) {
          s = 0;
          phase ^= 1;
        }
        issued = i + 1;
      }
      __syncwarp();
      if (*abort_flag) {
        volatile int never = 0;
        for (int i = max(0, issued - kStages); i < issued; ++i)
          mbar_wait(full_bar(i % kStages), (i / kStages) & 1, &never, nullptr, 0, kWaitTimeoutNs);
      }
    }
    return;
  }

  // ------------------------------------------------------------------ consumers
  const int t = static_cast<int>(threadIdx.x);  // 0..127
  // The row's queries, rotated, as the B operand's 16-bit terms. Sixteen threads
  // take a head: thread e elements 4e .. 4e+3.
  {
    const int hh = t >> 4, d0 = (t & 15) * 4;
#pragma unroll
    for (int tk = 0; tk < NT; ++tk) {
      float y[4] = {0.f, 0.f, 0.f, 0.f};
      if (t0 + tk < a.n && idx0 + tk >= 0) {
        int p = a.pos ? __ldg(a.pos + static_cast<int64_t>(b) * a.n + t0 + tk) : idx0 + tk;
        if (p < 0 || p >= kMaxPosition) {
          atomicOr(a.err, kErrPosition);
          p = p < 0 ? 0 : kMaxPosition - 1;
        }
        const uint16_t* q = a.q + b * a.q_batch + (t0 + tk) * a.q_token +
                            (g * kGroup + hh) * kHeadDim;
        const uint2 own = __ldg(reinterpret_cast<const uint2*>(q + d0));
        const uint2 other = __ldg(reinterpret_cast<const uint2*>(q + (d0 ^ 32)));
        const float4* cs = reinterpret_cast<const float4*>(
            a.rope + static_cast<int64_t>(p) * kRopePairs + (d0 & 31));
        const float4 c0 = __ldg(cs), c1 = __ldg(cs + 1);
        const float x[4] = {bf16lo_to_f32(own.x), bf16hi_to_f32(own.x), bf16lo_to_f32(own.y),
                            bf16hi_to_f32(own.y)};
        const float z[4] = {bf16lo_to_f32(other.x), bf16hi_to_f32(other.x),
                            bf16lo_to_f32(other.y), bf16hi_to_f32(other.y)};
        const float cc[4] = {c0.x, c0.z, c1.x, c1.z}, ss[4] = {c0.y, c0.w, c1.y, c1.w};
        const float sign = d0 < 32 ? -1.f : 1.f;
#pragma unroll
        for (int e = 0; e < 4; ++e) y[e] = fmaf(x[e], cc[e], sign * z[e] * ss[e]);
      }
      const uint32_t at = L::kQ + static_cast<uint32_t>((tk * kGroup + hh) * kHeadDim + d0) * 2;
      if (kFp8) {
        // largest element to [1, 2): f16 then holds the others to 2^-12 of themselves
        // or 2^-25 of the largest
        float top = fmaxf(fmaxf(fabsf(y[0]), fabsf(y[1])), fmaxf(fabsf(y[2]), fabsf(y[3])));
#pragma unroll
        for (int d = 8; d > 0; d /= 2) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
        int e = static_cast<int>(__float_as_uint(top) >> 23) - 127;
        e = max(-126, min(e, 126));
        const float f = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
        if (d0 == 0)
          *reinterpret_cast<float*>(smem + L::kQExp + (tk * kGroup + hh) * 4) =
              __uint_as_float(static_cast<uint32_t>(127 + e) << 23);
        *reinterpret_cast<uint2*>(smem + at) =
            make_uint2(pack_f16x2(y[0] * f, y[1] * f), pack_f16x2(y[2] * f, y[3] * f));
      } else {
        const uint32_t h0 = split_bf16x2(y[0], y[1]), h1 = split_bf16x2(y[2], y[3]);
        *reinterpret_cast<uint2*>(smem + at) = make_uint2(h0, h1);
        *reinterpret_cast<uint2*>(smem + at + NT * kGroup * kHeadDim * 2) =
            make_uint2(pack_bf16x2(y[0], y[1]), pack_bf16x2(y[2], y[3]));
      }
    }
  }
  named_barrier(1, kWarps * 32);

  const int gr = lane >> 2, tc = lane & 3;
  // B fragments of Q^T: column gr = head, rows 2tc, 2tc+1 and 2tc+8, 2tc+9 of k step kk.
  // e4m3: a lane's 16 bytes of a key are elements 16tc .. 16tc+15, four per k step, so
  // those rows stand for elements 16tc+4kk .. 16tc+4kk+3 (any order of the 64 will do).
  uint32_t qh[NT][4][2], ql[kFp8 ? 1 : NT][4][2];
  float qs[kFp8 ? NT : 1][2];
#pragma unroll
  for (int tk = 0; tk < NT; ++tk) {
    const uint8_t* q = smem + L::kQ + (tk * kGroup + gr) * kHeadDim * 2;
#pragma unroll
    for (int kk = 0; kk < 4; ++kk) {
      const int d0 = kFp8 ? 16 * tc + 4 * kk : 16 * kk + 2 * tc;
      const int d1 = kFp8 ? d0 + 2 : d0 + 8;
      qh[tk][kk][0] = *reinterpret_cast<const uint32_t*>(q + d0 * 2);
      qh[tk][kk][1] = *reinterpret_cast<const uint32_t*>(q + d1 * 2);
      if (!kFp8) {
        const uint8_t* q2 = q + NT * kGroup * kHeadDim * 2;
        ql[kFp8 ? 0 : tk][kk][0] = *reinterpret_cast<const uint32_t*>(q2 + d0 * 2);
        ql[kFp8 ? 0 : tk][kk][1] = *reinterpret_cast<const uint32_t*>(q2 + d1 * 2);
      }
    }
    if (kFp8) {
      const float2 e = *reinterpret_cast<const float2*>(smem + L::kQExp + (tk * kGroup + 2 * tc) * 4);
      qs[kFp8 ? tk : 0][0] = e.x;
      qs[kFp8 ? tk : 0][1] = e.y;
    }
  }

  // O^T of this warp's keys: four tiles of 16 head_dim rows; columns 2tc, 2tc+1 (heads).
  float o[NT][4][4], m[NT][2], l[NT][2];
#pragma unroll
  for (int tk = 0; tk < NT; ++tk) {
#pragma unroll
    for (int i = 0; i < 4; ++i) o[tk][i][0] = o[tk][i][1] = o[tk][i][2] = o[tk][i][3] = 0.f;
    m[tk][0] = m[tk][1] = kNoMax;
    l[tk][0] = l[tk][1] = 0.f;
  }
  // Keys that every token of the row sees need no mask.
  const int all_hi = idx0 + 1;  // keys below it are not past the first token
  const int all_lo = a.window > 0 ? min(idx0 + NT, len) - a.window : 0;
  // this lane's places in a block of 16 keys
  const uint32_t k_lane =
      kFp8 ? gr * 64 + ((tc ^ ((gr >> 1) & 3)) << 4) : (lane & 15) * 128;
  const int vr = kFp8 ? lane & 15 : (lane & 7) + 8 * (lane >> 4);  // key of a V matrix row
  bool ok = !skip;
  int s = 0;
  uint32_t phase = 0;
  for (int i = 0; ok && i < n_tiles; ++i) {
    if (!(ok = mbar_wait_warp(full_bar(s), phase, abort_flag, a.err, kErrTimeout, kWaitTimeoutNs)))
      break;
    const uint32_t block0 = static_cast<uint32_t>(16 * kBlocks * warp);
    const uint32_t sk = sbase + L::kK + s * kTileBytes + block0 * kRowBytes;
    const uint32_t sv = sbase + L::kV + s * kTileBytes + block0 * kRowBytes;
    const int key0 = key_a + i * kTile + static_cast<int>(block0);
    float4 pagef[kBlocks];
#pragma unroll
    for (int u = 0; u < kBlocks; ++u) {
      pagef[u] = make_float4(kScaleLog2, 0.f, 1.f, 0.f);
      if (kFp8)
        pagef[u] = *reinterpret_cast<const float4*>(
            smem + L::kPage + (s * L::kPages + kBlocks * warp + u) * 16);
    }

    // S^T: rows = keys gr and gr+8 of a block, columns = heads 2tc and 2tc+1
    float sc[kBlocks][NT][4];
#pragma unroll
    for (int u = 0; u < kBlocks; ++u) {
#pragma unroll
      for (int tk = 0; tk < NT; ++tk) sc[u][tk][0] = sc[u][tk][1] = sc[u][tk][2] = sc[u][tk][3] = 0.f;
      if (kFp8) {
        const uint4 ka = lds128(sk + k_lane + u * 1024);
        const uint4 kb = lds128(sk + k_lane + u * 1024 + 512);
        const uint32_t wa[4] = {ka.x, ka.y, ka.z, ka.w}, wb[4] = {kb.x, kb.y, kb.z, kb.w};
#pragma unroll
        for (int kk = 0; kk < 4; ++kk) {
          uint32_t f[4];
          e4m3x4_to_f16(wa[kk], f[0], f[2]);
          e4m3x4_to_f16(wb[kk], f[1], f[3]);
#pragma unroll
          for (int tk = 0; tk < NT; ++tk) mma_f16(sc[u][tk], f, qh[tk][kk][0], qh[tk][kk][1]);
        }
      } else {
#pragma unroll
        for (int kk = 0; kk < 4; ++kk) {
          uint32_t f[4];
          ldsm_x4(sk + k_lane + u * 2048 + (((2 * kk + (lane >> 4)) ^ (lane & 7)) << 4), f[0], f[1],
                  f[2], f[3]);
#pragma unroll
          for (int tk = 0; tk < NT; ++tk) {
            mma_bf16(sc[u][tk], f, qh[tk][kk][0], qh[tk][kk][1]);
            mma_bf16(sc[u][tk], f, ql[kFp8 ? 0 : tk][kk][0], ql[kFp8 ? 0 : tk][kk][1]);
          }
        }
      }
    }

    // Exponents x - m in log2 units; masked keys -inf.
    const bool edge = key0 + 16 * kBlocks > all_hi || key0 < all_lo;
    float d[kBlocks][NT][4], top = -INFINITY;
#pragma unroll
    for (int u = 0; u < kBlocks; ++u)
#pragma unroll
      for (int tk = 0; tk < NT; ++tk) {
        const float c0 = kFp8 ? pagef[u].x * qs[kFp8 ? tk : 0][0] : kScaleLog2;
        const float c1 = kFp8 ? pagef[u].x * qs[kFp8 ? tk : 0][1] : kScaleLog2;
        const float y0 = pagef[u].y - m[tk][0], y1 = pagef[u].y - m[tk][1];
        d[u][tk][0] = fmaf(sc[u][tk][0], c0, y0);
        d[u][tk][1] = fmaf(sc[u][tk][1], c1, y1);
        d[u][tk][2] = fmaf(sc[u][tk][2], c0, y0);
        d[u][tk][3] = fmaf(sc[u][tk][3], c1, y1);
        if (edge) {
          const int last = idx0 + tk, k0 = key0 + 16 * u + gr, k1 = k0 + 8;
          const int before = a.window > 0 ? last - a.window : -1;
          if (k0 > last || k0 <= before) d[u][tk][0] = d[u][tk][1] = -INFINITY;
          if (k1 > last || k1 <= before) d[u][tk][2] = d[u][tk][3] = -INFINITY;
        }
        top = fmax3(top, fmaxf(d[u][tk][0], d[u][tk][1]), fmaxf(d[u][tk][2], d[u][tk][3]));
      }
    if (__any_sync(0xffffffffu, top > kRescaleThreshold)) {
      // new maxima of every head, over the warp's keys
#pragma unroll
      for (int tk = 0; tk < NT; ++tk) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          float x[kBlocks][2], mx = m[tk][h];
#pragma unroll
          for (int u = 0; u < kBlocks; ++u) {
            const float c = kFp8 ? pagef[u].x * qs[kFp8 ? tk : 0][h] : kScaleLog2;
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              x[u][e] = fmaf(sc[u][tk][2 * e + h], c, pagef[u].y);
              if (d[u][tk][2 * e + h] != -INFINITY) mx = fmaxf(mx, x[u][e]);
            }
          }
#pragma unroll
          for (int w = 4; w < 32; w *= 2) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, w));
          const float alpha = ex2_approx(m[tk][h] - mx);
          m[tk][h] = mx;
          l[tk][h] *= alpha;
#pragma unroll
          for (int mt = 0; mt < 4; ++mt) {
            o[tk][mt][h] *= alpha;
            o[tk][mt][2 + h] *= alpha;
          }
#pragma unroll
          for (int u = 0; u < kBlocks; ++u)
#pragma unroll
            for (int e = 0; e < 2; ++e)
              if (d[u][tk][2 * e + h] != -INFINITY) d[u][tk][2 * e + h] = x[u][e] - mx;
        }
      }
    }

    // P^T, transposed to the B operand (row = key, column = head)
    uint32_t ph[kBlocks][NT][2], pl[kBlocks][kFp8 ? 1 : NT][2];
#pragma unroll
    for (int u = 0; u < kBlocks; ++u)
#pragma unroll
      for (int tk = 0; tk < NT; ++tk) {
        float p[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) p[e] = ex2_approx(d[u][tk][e]);
        l[tk][0] = fmaf(p[0] + p[2], pagef[u].z, l[tk][0]);
        l[tk][1] = fmaf(p[1] + p[3], pagef[u].z, l[tk][1]);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          if (kFp8) {
            ph[u][tk][h] = transpose8(pack_f16x2(p[2 * h], p[2 * h + 1]));
          } else {
            ph[u][tk][h] = transpose8(split_bf16x2(p[2 * h], p[2 * h + 1]));
            pl[u][kFp8 ? 0 : tk][h] = transpose8(pack_bf16x2(p[2 * h], p[2 * h + 1]));
          }
        }
      }

    // O^T += V^T P^T
#pragma unroll
    for (int u = 0; u < kBlocks; ++u) {
      auto accumulate = [&](int mt, const uint32_t (&f)[4]) {
#pragma unroll
        for (int tk = 0; tk < NT; ++tk) {
          uint32_t z[4] = {f[0], f[1], f[2], f[3]};
          if (edge) {
            // the values of this token's masked keys are zeroed: their p is 0, but what lies
            // there may be infinite or NaN
            const int last = idx0 + tk, before = a.window > 0 ? last - a.window : -1;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const int k0 = key0 + 16 * u + 8 * h + 2 * tc;
              const uint32_t keep = (k0 <= last && k0 > before ? 0x0000FFFFu : 0u) |
                                    (k0 + 1 <= last && k0 + 1 > before ? 0xFFFF0000u : 0u);
              z[2 * h] &= keep;
              z[2 * h + 1] &= keep;
            }
          }
          if (kFp8) {
            mma_f16(o[tk][mt], z, ph[u][tk][0], ph[u][tk][1]);
          } else {
            mma_bf16(o[tk][mt], z, ph[u][tk][0], ph[u][tk][1]);
            mma_bf16(o[tk][mt], z, pl[u][kFp8 ? 0 : tk][0], pl[u][kFp8 ? 0 : tk][1]);
          }
        }
      };
      if (kFp8) {
        // a lane's word: keys 2tc, 2tc+1 of elements 16c+2gr, 16c+2gr+1; rows gr and
        // gr+8 of tile c stand for those two
#pragma unroll
        for (int c = 0; c < 4; c += 2) {
          uint32_t w[4];
          ldsm_x4_trans(sv + u * 1024 + vr * 64 + (((c + (lane >> 4)) ^ ((vr >> 1) & 3)) << 4), w[0],
                        w[1], w[2], w[3]);
#pragma unroll
          for (int v = 0; v < 2; ++v) {
            uint32_t f[4];
            e4m3x4_to_f16(__byte_perm(w[2 * v], 0, 0x3120), f[0], f[1]);
            e4m3x4_to_f16(__byte_perm(w[2 * v + 1], 0, 0x3120), f[2], f[3]);
            accumulate(c + v, f);
          }
        }
      } else {
#pragma unroll
        for (int mt = 0; mt < 4; ++mt) {
          uint32_t f[4];
          ldsm_x4_trans(
              sv + u * 2048 + vr * 128 + (((2 * mt + ((lane >> 3) & 1)) ^ (vr & 7)) << 4), f[0],
              f[1], f[2], f[3]);
          accumulate(mt, f);
        }
      }
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(empty_bar(s));
    if (++s == kStages) {
      s = 0;
      phase ^= 1;
    }
  }

  // ---- join the warps
  named_barrier(1, kWarps * 32);  // every warp has done with the tiles
  if (kFp8 && *far) {
    if (skip || *abort_flag) return;
    const int tokens = min(NT, a.n - t0);
#pragma unroll 1
    for (int i = 2 * warp + (lane >> 4); i < tokens * kGroup; i += 2 * kWarps)
      plain_row(a, b, t0 + i / kGroup, idx0 + i / kGroup, g * kGroup + i % kGroup, key_a,
                key_a + n_tiles * kTile, chunks,
                (static_cast<int64_t>(part) * kNumKvHeads + g) * (NT * kGroup) + i);
    return;
  }
  float* mo = reinterpret_cast<float*>(smem + L::kMerge + warp * L::kMergeWarp);
#pragma unroll
  for (int tk = 0; tk < NT; ++tk)
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      float* row_o = mo + (tk * kGroup + 2 * tc + h) * kHeadDim;
#pragma unroll
      for (int mt = 0; mt < 4; ++mt) {
        row_o[16 * mt + (kFp8 ? 2 * gr : gr)] = o[tk][mt][h];
        row_o[16 * mt + (kFp8 ? 2 * gr + 1 : gr + 8)] = o[tk][mt][2 + h];
      }
      float sum = l[tk][h];
#pragma unroll
      for (int w = 4; w < 32; w *= 2) sum += __shfl_xor_sync(0xffffffffu, sum, w);
      if (gr == 0) {
        float* ml = mo + NT * kGroup * kHeadDim;
        ml[tk * kGroup + 2 * tc + h] = m[tk][h];
        ml[NT * kGroup + tk * kGroup + 2 * tc + h] = sum;
      }
    }
  named_barrier(1, kWarps * 32);
  if (skip || *abort_flag) return;
  const int hh = t >> 4, d0 = (t & 15) * 4;
#pragma unroll
  for (int tk = 0; tk < NT; ++tk) {
    if (t0 + tk >= a.n) break;
    const int r = tk * kGroup + hh;
    float mw[kWarps], M = kNoMax;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const float* base = reinterpret_cast<const float*>(smem + L::kMerge + w * L::kMergeWarp);
      mw[w] = base[NT * kGroup * kHeadDim + r];
      M = fmaxf(M, mw[w]);
    }
    float sum = 0.f, acc[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const float* base = reinterpret_cast<const float*>(smem + L::kMerge + w * L::kMergeWarp);
      const float f = ex2_approx(mw[w] - M);
      sum = fmaf(f, base[NT * kGroup * (kHeadDim + 1) + r], sum);
      const float4 v = *reinterpret_cast<const float4*>(base + r * kHeadDim + d0);
      acc[0] = fmaf(f, v.x, acc[0]);
      acc[1] = fmaf(f, v.y, acc[1]);
      acc[2] = fmaf(f, v.z, acc[2]);
      acc[3] = fmaf(f, v.w, acc[3]);
    }
    if (chunks == 1) {
      const float sink = __ldg(a.sinks + g * kGroup + hh) * kLog2e;
      const float Mf = fmaxf(sink, M);
      const float f = ex2_approx(M - Mf);
      const float den = fmaf(f, sum, ex2_approx(sink - Mf));
      const float scale = M > kNoMax ? f / den : 0.f;
      const float grow = kFp8 ? paged_power(*unit) : 1.f;
      *reinterpret_cast<uint2*>(
          a.out + ((static_cast<int64_t>(b) * a.n + t0 + tk) * kNumHeads + g * kGroup + hh) *
                      kHeadDim + d0) =
          make_uint2(pack_bf16x2(acc[0] * scale * grow, acc[1] * scale * grow),
                     pack_bf16x2(acc[2] * scale * grow, acc[3] * scale * grow));
    } else {
      if (kFp8) {
        const float2 f = to_part(&M, &sum, *unit);
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[e] = acc[e] * f.x * f.y;
      }
      const int64_t pr = (static_cast<int64_t>(part) * kNumKvHeads + g) * (NT * kGroup) + r;
      *reinterpret_cast<float4*>(a.part_o + pr * kHeadDim + d0) =
          make_float4(acc[0], acc[1], acc[2], acc[3]);
      if (d0 == 0) a.part_ml[pr] = make_float2(M, sum);
    }
  }
}

template <bool kFp8, int NT>
cudaError_t launch(const PagedMaps& maps, const PagedAttentionArgs& a, cudaStream_t stream) {
  using L = Smem<kFp8, NT>;
  static std::atomic<uint64_t> prepared{0};  // devices whose kernel has its shared memory
  cudaError_t e = allow_shared(reinterpret_cast<const void*>(paged_attention_kernel<kFp8, NT>), L::kBytes,
                               &prepared);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cfg.stream = stream;
  const int64_t chunks = paged_max_chunks(a.rows, a.most, a.target);
  cfg.gridDim = dim3(static_cast<unsigned>(chunks * kNumKvHeads));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = L::kBytes;
  e = cudaLaunchKernelEx(&cfg, paged_attention_kernel<kFp8, NT>, maps, a);
  if (e != cudaSuccess || a.none_cut) return e;
  return launch_paged_combine(a, NT, stream);
}

}  // namespace

cudaError_t launch_paged_attention(const PagedMaps& maps, const PagedAttentionArgs& a,
                                   cudaStream_t stream) {
  switch (paged_row_tokens(a.n)) {
    case 1: return a.cache.fp8 ? launch<true, 1>(maps, a, stream) : launch<false, 1>(maps, a, stream);
    case 2: return a.cache.fp8 ? launch<true, 2>(maps, a, stream) : launch<false, 2>(maps, a, stream);
    default: return launch_paged_attention_many(maps, a, stream);
  }
}

}  // namespace gqa
