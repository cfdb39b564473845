// Attention over a paged key/value cache for rows of many query tokens (drafts, a piece
// of a prompt on a cached prefix), on the 5th-generation tensor cores of sm_100a.
//
// A row is 16 consecutive query tokens of one sequence; with the 8 query heads of a
// group they are the 128 rows of tcgen05.mma, S = Q K^T and O += P V with fp32 in
// tensor memory. Work is cut as for few tokens (paged.h): rows by tiles of 128 keys,
// rows of many tiles into chunks that the combine kernel joins.
//
// A CTA has two halves of 256 threads, which take two kv heads of the same chunk, each
// with its own pipeline. Their softmax warps take turns at the exponential unit: left
// alone (as two CTAs of an SM) they fall into step, use it together and then leave it
// idle together. Roles in a half:
//   warps 0-3  softmax, one thread per query row (TMEM lane): rotate and store Q, then
//              per tile load S (128 columns), exponentials, P to TMEM; at the end O.
//              Warps whose four tokens are past the row's last take no part.
//   warp 4     producer: pages to shared memory (TMA)
//   warp 5     issues the products (of the first half: owns the tensor memory)
//   warps 6-7  look over the value rows of tiles at the edge; e4m3: codes to f16, K and V
//              of a tile each into its own buffer
//
// Precision. bf16 pages: q in two bf16 terms (two products), p in one (2^-8, as in the prefill
// kernels: a second term of p has no room beside S and O of both halves in tensor memory, and
// its store and product would lengthen the chain that bounds the loop). e4m3
// pages: codes are exact in f16, and q, scaled by a power of two, and p are f16 (2^-12
// each); scales of pages enter per 16 columns, in the chunk's unit, as in the kernel for few
// tokens.
//
// Masked values. P is 0 where a query does not see a key, but 0 * NaN is NaN, and in a
// tile at the edge of what is visible the value rows may be stale or belong to later
// tokens. There, value rows that no token of the row sees, or that hold an infinity
// or NaN, are zeroed in shared memory; the latter are noted, and the softmax warps add
// them to the queries that see them one by one (exact, and as slow as it is rare).
//
// The floor of whole rows is the exponential unit: 128 x 128 of them per tile take 1024
// cycles of an SM. A pair of halves takes about 3800 for its two tiles, as a row's thread has
// its loads, maximum, exponentials and stores one after the other and only the other
// half's beside them: 512 tokens on 4096 cached ones take 79 us (bf16; 464 TFLOP/s) and 90
// (e4m3), of which 32 chunks of 33 to 36 tiles on 37 places. Before the first tile a CTA
// spends about 5.5 us. Two threads per row, of 64 columns each, which tell each other
// their maximum, took 96 to 114 us.
#include "paged_common.cuh"

namespace gqa {
namespace {

constexpr int kNT = kPagedManyTokens;
constexpr int kTile = kPagedTileN;
constexpr int kHalf = 256;  // threads of a half
constexpr int kThreads = 2 * kHalf;
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kHalfCols = 256;  // S [0,128), P [128,192), O [192,256)
constexpr uint32_t kColP = 128, kColO = 192;
constexpr uint32_t kTile16 = kTile * kHeadDim * 2;  // a tile of 16-bit elements
constexpr uint32_t kTile8 = kTile * kHeadDim;

constexpr uint32_t kRegsLight = 72;
constexpr uint32_t kRegsSoftmax = 184;
static_assert(256 * kRegsLight + 256 * kRegsSoftmax <= 512 * 128, "register split");

// Exp-loop step (of 64 column pairs) at which a softmax warp lets the other half's go on
// (22: 77.9 us, 30: 78.8, 38: 79.1 for 512 bf16 tokens on 4096; 2 to 18 were no better).
constexpr int kTurnHandOff = 22;
constexpr int kAskPv = 56;  // step at which it asks for the products of the tile before

constexpr int kRaw = 3;    // stages of e4m3 tiles
constexpr int kPageRing = 4;  // tiles whose pages' factors are held: written by the producer up
                              // to kRaw tiles ahead of the softmax

// A half's shared memory; then what the CTA shares.
template <bool kFp8>
struct Smem {
  static constexpr int kStages = kFp8 ? 1 : 2;  // of the 16-bit operands
  static constexpr uint32_t kQ = 0;             // [terms] 128 rows
  static constexpr uint32_t kK = kQ + (kFp8 ? 1 : 2) * kTile16;
  static constexpr uint32_t kV = kK + kStages * kTile16;
  static constexpr uint32_t kRawK = kV + kStages * kTile16;
  static constexpr uint32_t kRawV = kRawK + (kFp8 ? kRaw : 0) * kTile8;
  static constexpr uint32_t kPage = kRawV + (kFp8 ? kRaw : 0) * kTile8;  // float4 [ring][8]
  static constexpr uint32_t kBar = kPage + (kFp8 ? kPageRing * 8 * 16 : 0);
  static constexpr uint32_t kBad = kBar + 32 * 8;  // [2][2][4] value rows taken out of a tile
  static constexpr uint32_t kUnit = kBad + 64;  // e4m3: whether a value scale lies too far from
                                                // the chunk's unit; that unit
  static constexpr uint32_t kHalfBytes = (kUnit + 8 + 1023) / 1024 * 1024;
  static constexpr uint32_t kScan = 2 * kHalfBytes;  // 16 + 16 warp sums, slot
  static constexpr uint32_t kMisc = kScan + 32 * 4 + sizeof(ScanSlot);  // abort flag, TMEM address
  static constexpr uint32_t kBytes = kMisc + 16 + 1024;
};
static_assert(Smem<false>::kBytes <= 227 * 1024 && Smem<true>::kBytes <= 227 * 1024, "shared memory");

enum : int {
  BAR_Q = 0,        // Q stored and O zeroed
  BAR_S_FULL,       // S of a tile written (and its K free)
  BAR_S_FREE,       // S loaded by the softmax
  BAR_P_FULL,       // P written
  BAR_PV,           // P V done: P and the tile's V free, O complete so far
  BAR_DONE,         // every product done (exit)
  BAR_K_FULL,       // [2] bf16: tile loaded; e4m3: [0] tile converted
  BAR_V_FULL = BAR_K_FULL + 2,
  BAR_K_FREE = BAR_V_FULL + 2,  // [2] bf16
  BAR_V_FREE = BAR_K_FREE + 2,
  BAR_RAW = BAR_V_FREE + 2,     // [kRaw] e4m3: tile loaded
  BAR_RAW_FREE = BAR_RAW + kRaw,
  BAR_SEEN = BAR_RAW_FREE + kRaw,  // [2] value rows of a tile at the edge looked over
  BAR_TURN = BAR_SEEN + 2,         // [4] softmax warp w may use the exponential unit
  NUM_BARS = BAR_TURN + 4
};
static_assert(NUM_BARS <= 32, "barriers");

// Instruction descriptor, kind::f16, fp32 accumulators.
template <bool kFp8>
__host__ __device__ constexpr uint32_t idesc(int N, bool b_mn_major) {
  return idesc_bf16(128, N, b_mn_major) & (kFp8 ? ~((7u << 7) | (7u << 10)) : ~0u);
}

// One column of this thread's lane, waited on.
__device__ __forceinline__ float tmem_ld1(uint32_t taddr) {
  uint32_t r;
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x1.b32 {%0}, [%1];\n\ttcgen05.wait::ld.sync.aligned;"
               : "=r"(r)
               : "r"(taddr)
               : "memory");
  return __uint_as_float(r);
}

// Whether a word of two 16-bit floats holds an infinity or NaN.
template <bool kFp8>
__device__ __forceinline__ bool not_finite(uint32_t w) {
  constexpr uint32_t m = kFp8 ? 0x7C00u : 0x7F80u;
  return (w & m) == m || ((w >> 16) & m) == m;
}

struct Ctx {
  uint32_t sbase, bars;
  volatile int* abort_flag;
  int* err;
  __device__ uint32_t bar(int i) const { return bars + 8u * static_cast<uint32_t>(i); }
  __device__ bool wait(int i, uint32_t parity) const {
    return mbar_wait(bar(i), parity, abort_flag, err, kErrTimeout, kWaitTimeoutNs);
  }
  // Whether the phase is over already, asked ahead of the wait so that the answer's latency
  // passes under other work; for wait_asked.
  __device__ uint32_t ask(int i, uint32_t parity) const { return mbar_test_wait(bar(i), parity); }
  __device__ bool wait_asked(uint32_t over, int i, uint32_t parity) const {
    return __all_sync(0xffffffffu, over) || wait_warp(i, parity);
  }
  __device__ bool wait_warp(int i, uint32_t parity) const {
    return mbar_wait_warp(bar(i), parity, abort_flag, err, kErrTimeout, kWaitTimeoutNs);
  }
};

// Rotates this thread's query row, splits or scales it to 16 bits and stores it as row r
// of the Q operand (zeros if there is no such token). Returns the power of two
// that an e4m3 row was divided by.
template <bool kFp8>
__device__ __forceinline__ float store_query(const PagedAttentionArgs& a, uint8_t* smem, int b,
                                             int t, int idx, int head, int r) {
  float y[64];
#pragma unroll
  for (int e = 0; e < 64; ++e) y[e] = 0.f;
  if (t < a.n && idx >= 0) {
    int p = a.pos ? __ldg(a.pos + static_cast<int64_t>(b) * a.n + t) : idx;
    if (p < 0 || p >= kMaxPosition) {
      atomicOr(a.err, kErrPosition);
      p = p < 0 ? 0 : kMaxPosition - 1;
    }
    const uint4* q4 = reinterpret_cast<const uint4*>(a.q + b * a.q_batch + t * a.q_token +
                                                     head * kHeadDim);
    const float4* cs = reinterpret_cast<const float4*>(a.rope + static_cast<int64_t>(p) * kRopePairs);
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      const uint4 lo = __ldg(q4 + c), hi = __ldg(q4 + c + 4);
      const uint32_t lw[4] = {lo.x, lo.y, lo.z, lo.w}, hw[4] = {hi.x, hi.y, hi.z, hi.w};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float4 f = __ldg(cs + 4 * c + e);  // (cos, sin) of two pairs
        const float l0 = bf16lo_to_f32(lw[e]), l1 = bf16hi_to_f32(lw[e]);
        const float h0 = bf16lo_to_f32(hw[e]), h1 = bf16hi_to_f32(hw[e]);
        const int d = 8 * c + 2 * e;
        y[d] = fmaf(l0, f.x, -h0 * f.y);
        y[d + 1] = fmaf(l1, f.z, -h1 * f.w);
        y[d + 32] = fmaf(h0, f.x, l0 * f.y);
        y[d + 33] = fmaf(h1, f.z, l1 * f.w);
      }
    }
  }
  float unit = 1.f, f = 1.f;
  if (kFp8) {
    float top = 0.f;
#pragma unroll
    for (int e = 0; e < 64; ++e) top = fmaxf(top, fabsf(y[e]));
    int e = static_cast<int>(__float_as_uint(top) >> 23) - 127;
    e = max(-126, min(e, 126));
    f = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
    unit = __uint_as_float(static_cast<uint32_t>(127 + e) << 23);
  }
  uint8_t* row = smem + Smem<kFp8>::kQ + r * 128;  // of this half
#pragma unroll
  for (int c = 0; c < 8; ++c) {
    uint32_t w[4], v[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      float y0 = y[8 * c + 2 * e], y1 = y[8 * c + 2 * e + 1];
      if (kFp8) {
        w[e] = pack_f16x2(y0 * f, y1 * f);
      } else {
        w[e] = split_bf16x2(y0, y1);
        v[e] = pack_bf16x2(y0, y1);
      }
    }
    uint8_t* at = row + ((c ^ (r & 7)) << 4);
    *reinterpret_cast<uint4*>(at) = make_uint4(w[0], w[1], w[2], w[3]);
    if (!kFp8) *reinterpret_cast<uint4*>(at + kTile16) = make_uint4(v[0], v[1], v[2], v[3]);
  }
  return unit;
}

template <bool kFp8>
__global__ void __launch_bounds__(kThreads, 1)
    paged_many_kernel(const __grid_constant__ PagedMaps maps, const PagedAttentionArgs a) {
  using L = Smem<kFp8>;
  constexpr uint32_t kRowBytes = kHeadDim * (kFp8 ? 1 : 2);
  griddep_launch_dependents();
  if (threadIdx.x == 4 * 32) {
    prefetch_tensormap(&maps.k);
    prefetch_tensormap(&maps.v);
  }
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  const int half = static_cast<int>(threadIdx.x / kHalf);
  uint8_t* cta_smem = smem;
  smem += half * L::kHalfBytes;  // this half's
  Ctx ctx;
  ctx.sbase = smem_u32(smem);
  ctx.bars = ctx.sbase + L::kBar;
  ctx.abort_flag = reinterpret_cast<volatile int*>(cta_smem + L::kMisc);
  ctx.err = a.err;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(cta_smem + L::kMisc + 4);
  const int ht = static_cast<int>(threadIdx.x % kHalf);  // thread and warp of the half
  const int warp = ht >> 5;
  const int lane = ht & 31;
  volatile int* far = reinterpret_cast<volatile int*>(smem + L::kUnit);
  volatile int* unit_of = far + 1;
  constexpr int kCtas = kNumKvHeads / 2;  // of a chunk
  const int g = static_cast<int>(blockIdx.x % kCtas) * 2 + half;

  // The tokens, lengths and pages, the workspace and the tensor memory may still be in
  // use by the kernel before.
  griddep_wait();
  if (threadIdx.x == 0)
    *ctx.abort_flag = (*reinterpret_cast<volatile int*>(a.err) & kErrTimeout) ? 1 : 0;
  ScanSlot* slot = reinterpret_cast<ScanSlot*>(cta_smem + L::kScan + 32 * 4);
  if (!find_chunk<kNT, kTile, kThreads>(a, static_cast<int>(blockIdx.x / kCtas),
                                        reinterpret_cast<uint32_t*>(cta_smem + L::kScan), slot))
    return;  // past the call's last chunk
  const bool skip = *ctx.abort_flag != 0;
  const int row = slot->row, chunks = slot->chunks, part = slot->part + slot->split;
  if (a.meta && slot->split == 0 && g == 0 && threadIdx.x == 0)
    a.meta[row] = make_int2(slot->part, chunks);
  const int b = sequence_of(a, row);
  const int t0 = (row - b * a.groups) * kNT;
  const int len = slot->len;
  const int idx0 = len - a.n + t0;  // index of the row's first token
  int lo, hi, tile_a, tile_b;
  paged_row_range(len, a.n, t0, kNT, a.window, &lo, &hi);
  paged_chunk_range(paged_row_tiles(lo, hi, kTile), chunks, slot->split, &tile_a, &tile_b);
  const int key_a = (lo / kTile + tile_a) * kTile;  // first key of the chunk's tiles
  const int n_tiles = tile_b - tile_a;
  const int active = (min(kNT, a.n - t0) + 3) / 4;  // softmax warps with tokens
  const int page_log2 = a.cache.page_log2;
  const int32_t* table = a.table + static_cast<int64_t>(b) * a.max_pages;

  // Keys from edge_hi on, or below edge_lo, are masked for some token of the row.
  const int edge_lo = a.window > 0 ? min(idx0 + kNT, len) - a.window : 0;
  const int edge_hi = idx0 + 1;
  auto at_edge = [&](int j) {
    const int key0 = key_a + j * kTile;
    return key0 + kTile > edge_hi || key0 < edge_lo;
  };

  if (warp >= 4) {
    setmaxnreg_dec<kRegsLight>();
    // Barriers and tensor memory, for these warps now and for the softmax warps (barrier 1)
    // when they have stored Q.
    if (ht == kHalf / 2) {
      const uint32_t warps = static_cast<uint32_t>(active);
      mbar_init(ctx.bar(BAR_Q), 32 * warps);
      mbar_init(ctx.bar(BAR_S_FULL), 1);
      mbar_init(ctx.bar(BAR_S_FREE), warps);
      mbar_init(ctx.bar(BAR_P_FULL), warps);
      mbar_init(ctx.bar(BAR_PV), 1);
      mbar_init(ctx.bar(BAR_DONE), 1);
      for (int i = 0; i < 2; ++i) {
        mbar_init(ctx.bar(BAR_K_FULL + i), kFp8 ? 64 : 1);
        mbar_init(ctx.bar(BAR_V_FULL + i), kFp8 ? 64 : 1);
        mbar_init(ctx.bar(BAR_K_FREE + i), 1);
        mbar_init(ctx.bar(BAR_V_FREE + i), 3);  // the products, warps 6 and 7
        mbar_init(ctx.bar(BAR_SEEN + i), 64);
      }
      for (int i = 0; i < 4; ++i) mbar_init(ctx.bar(BAR_TURN + i), 1);
      for (int i = 0; i < kRaw; ++i) {
        mbar_init(ctx.bar(BAR_RAW + i), 1);
        mbar_init(ctx.bar(BAR_RAW_FREE + i), 64);
      }
      fence_barrier_init();
      *far = *unit_of = 0;
    }
    if (half == 0 && warp == 5) {
      tmem_alloc(smem_u32(tmem_slot), kTmemCols);
      tmem_relinquish();
    }
    tc_fence_before_sync();
    named_barrier(2, kThreads / 2);
    tc_fence_after_sync();
    named_arrive(1, kThreads);
    const uint32_t tmem = *tmem_slot + half * kHalfCols;
    if (warp == 4 && !skip) {
      // ---------------------------------------------------------------- producer
      const int P = 1 << page_log2;
      const int box = P < kPagedTile ? P : kPagedTile;  // keys per copy
      const int boxes = kTile / box;                    // 2, 4 or 8
      const int last_page = (hi - 1) >> page_log2;
      auto fetch = [&](int pi) { return fetch_page<kFp8>(a, table, pi, lo, last_page, g); };
      int pbase = key_a >> page_log2;
      PageEntry cur = {}, nxt = {};
      if (n_tiles > 0) {
        cur = fetch(pbase + lane);
        nxt = fetch(pbase + 32 + lane);
      }
      int in = 0;  // the chunk's unit
      if (kFp8 && n_tiles > 0) {
        in = paged_unit(__shfl_sync(0xffffffffu, cur.vs, (max(key_a, lo) >> page_log2) - pbase));
        if (lane == 0) *unit_of = in;
      }
      const int sub = lane & 7;
      int issued_k = 0, issued_v = 0;
      for (int i = 0; i < n_tiles; ++i) {
        const int key0 = key_a + i * kTile;
        if ((key0 >> page_log2) >= pbase + 32) {
          pbase += 32;
          cur = nxt;
          nxt = fetch(pbase + 32 + lane);
        }
        const int s = i % (kFp8 ? kRaw : 2);
        const uint32_t round = static_cast<uint32_t>(i / (kFp8 ? kRaw : 2));
        if (round > 0 &&
            !ctx.wait_warp((kFp8 ? BAR_RAW_FREE : BAR_K_FREE) + s, (round - 1) & 1))
          break;
        // pages of this tile that hold a visible key
        const int key = key0 + sub * box;
        const int page = __shfl_sync(0xffffffffu, cur.page, ((key >> page_log2) - pbase) & 31);
        const bool load = sub < boxes && key < hi && key + box > lo;
        const uint32_t bytes =
            static_cast<uint32_t>(__popc(__ballot_sync(0xffffffffu, load) & 0xFFu) * box) * kRowBytes;
        if (kFp8) {
          if (lane == 0) mbar_expect_tx(ctx.bar(BAR_RAW + s), 2 * bytes);
          __syncwarp();
          if (load && lane < 16)
            tma_load_4d(ctx.sbase + (lane < 8 ? L::kRawK : L::kRawV) + s * kTile8 +
                            static_cast<uint32_t>(sub * box) * kRowBytes,
                        lane < 8 ? &maps.k : &maps.v, ctx.bar(BAR_RAW + s), 0, g, key & (P - 1),
                        page);
          const int pw = (key0 + sub * 16) >> page_log2;  // page of 16 columns
          const float ks = __shfl_sync(0xffffffffu, cur.ks, (pw - pbase) & 31);
          const float vs = __shfl_sync(0xffffffffu, cur.vs, (pw - pbase) & 31);
          if (lane < 8)
            *reinterpret_cast<float4*>(smem + L::kPage + ((i % kPageRing) * 8 + lane) * 16) =
                page_factors(ks, vs, in, far);
          __syncwarp();
          if (lane == 0) mbar_arrive(ctx.bar(BAR_RAW + s));  // and the scales are there
          issued_k = i + 1;
        } else {
          if (lane == 0) mbar_arrive_expect_tx(ctx.bar(BAR_K_FULL + s), bytes);
          __syncwarp();
          const uint32_t at = s * kTile16 + static_cast<uint32_t>(sub * box) * kRowBytes;
          if (load && lane < 8)
            tma_load_4d(ctx.sbase + L::kK + at, &maps.k, ctx.bar(BAR_K_FULL + s), 0, g,
                        key & (P - 1), page);
          issued_k = i + 1;
          if (round > 0 && !ctx.wait_warp(BAR_V_FREE + s, (round - 1) & 1)) break;
          if (lane == 0) mbar_arrive_expect_tx(ctx.bar(BAR_V_FULL + s), bytes);
          __syncwarp();
          if (load && lane < 8)
            tma_load_4d(ctx.sbase + L::kV + at, &maps.v, ctx.bar(BAR_V_FULL + s), 0, g,
                        key & (P - 1), page);
          issued_v = i + 1;
        }
      }
      __syncwarp();
      if (*ctx.abort_flag) {
        // Let every copy land before shared memory is released.
        volatile int never = 0;
        const int ring = kFp8 ? kRaw : 2;
        for (int i = max(0, issued_k - ring); i < issued_k; ++i)
          mbar_wait(ctx.bar((kFp8 ? BAR_RAW : BAR_K_FULL) + i % ring), (i / ring) & 1, &never,
                    nullptr, 0, kWaitTimeoutNs);
        for (int i = max(0, issued_v - ring); i < issued_v; ++i)
          mbar_wait(ctx.bar(BAR_V_FULL + i % ring), (i / ring) & 1, &never, nullptr, 0,
                    kWaitTimeoutNs);
      }
    } else if (warp == 5 && !skip && lane == 0 && n_tiles > 0) {
      // ---------------------------------------------------------------- products
      constexpr uint32_t kIdescQK = idesc<kFp8>(kTile, false);
      constexpr uint32_t kIdescPV = idesc<kFp8>(kHeadDim, true);
      auto issue_qk = [&](int j) {
        const int s = kFp8 ? 0 : j & 1;
        if (!ctx.wait(BAR_K_FULL + s, (kFp8 ? j : j >> 1) & 1)) return false;
        if (j > 0 && !ctx.wait(BAR_S_FREE, (j - 1) & 1)) return false;
        tc_fence_after_sync();
        const uint64_t ka = sdesc_sw128(ctx.sbase + L::kK + s * kTile16);
#pragma unroll
        for (int term = 0; term < (kFp8 ? 1 : 2); ++term) {
          const uint64_t qa = sdesc_sw128(ctx.sbase + L::kQ + term * kTile16);
#pragma unroll
          for (int kk = 0; kk < kHeadDim / 16; ++kk)  // 32 bytes along K
            mma_bf16_ss(tmem, qa + 2 * kk, ka + 2 * kk, kIdescQK, term + kk > 0 ? 1u : 0u);
        }
        mma_commit(ctx.bar(BAR_S_FULL));
        if (!kFp8) mma_commit(ctx.bar(BAR_K_FREE + s));
        return true;
      };
      uint32_t edges = 0;  // tiles at the edge so far
      auto issue_pv = [&](int j) {
        const int s = kFp8 ? 0 : j & 1;
        if (!ctx.wait(BAR_V_FULL + s, (kFp8 ? j : j >> 1) & 1) || !ctx.wait(BAR_P_FULL, j & 1))
          return false;
        if (!kFp8 && at_edge(j)) {
          if (!ctx.wait(BAR_SEEN + (edges & 1), (edges >> 1) & 1)) return false;
          ++edges;
        }
        tc_fence_after_sync();
        const uint64_t va = sdesc_sw128(ctx.sbase + L::kV + s * kTile16);
#pragma unroll
        for (int kk = 0; kk < kTile / 16; ++kk)  // 16 keys: two 8-row groups
          mma_bf16_ts(tmem + kColO, tmem + kColP + 8 * kk, va + 128 * kk, kIdescPV, 1u);
        mma_commit(ctx.bar(BAR_PV));
        if (!kFp8) mma_commit(ctx.bar(BAR_V_FREE + s));
        return true;
      };
      bool ok = ctx.wait(BAR_Q, 0) && issue_qk(0);
      for (int j = 0; ok && j < n_tiles; ++j)
        ok = (j + 1 == n_tiles || issue_qk(j + 1)) && issue_pv(j);
      // Every product issued must finish before the tensor memory is released.
      mma_commit(ctx.bar(BAR_DONE));
      volatile int never = 0;
      mbar_wait(ctx.bar(BAR_DONE), 0, &never, nullptr, 0, kWaitTimeoutNs);
    } else if (warp >= 6 && !skip) {
      // ---------------------------------------------------------------- value rows; e4m3 to f16
      const int t = ht - 192;  // 0..63
      uint32_t edges = 0;      // tiles at the edge so far
      uint32_t* bad_rows = reinterpret_cast<uint32_t*>(smem + L::kBad) + 4 * (t >> 5);  // this warp's
      // Four lanes look over a row each time, for whether it stays; the row's lanes agree.
      auto row_stays = [&](int j, int row_, bool finite) {
        const int key = key_a + j * kTile + row_;
        const bool seen = key >= lo && key < hi;
        const uint32_t all = __ballot_sync(0xffffffffu, finite);
        const bool fine = ((all >> (lane & 28)) & 0xFu) == 0xFu;
        if (seen && !fine && (lane & 3) == 0)
          atomicOr(bad_rows + 8 * (edges & 1) + (row_ >> 5), 1u << (row_ & 31));
        return seen && fine;
      };
      auto clear_bad = [&] {
        if (lane < 4) bad_rows[8 * (edges & 1) + lane] = 0u;
        __syncwarp();
      };
      // one tile of codes (64-byte rows, 64-byte swizzle) to f16 (128-byte rows and swizzle)
      auto convert = [&](uint32_t src, uint32_t dst, bool look, int j) {
#pragma unroll 2
        for (int i = t; i < kTile * 4; i += 64) {
          const int r = i >> 2, c = i & 3;
          const uint4 w = lds128(src + r * 64 + ((c ^ ((r >> 1) & 3)) << 4));
          uint4 x, y;
          e4m3x4_to_f16(w.x, x.x, x.y);
          e4m3x4_to_f16(w.y, x.z, x.w);
          e4m3x4_to_f16(w.z, y.x, y.y);
          e4m3x4_to_f16(w.w, y.z, y.w);
          if (look) {
            const bool finite = !(not_finite<true>(x.x) || not_finite<true>(x.y) ||
                                  not_finite<true>(x.z) || not_finite<true>(x.w) ||
                                  not_finite<true>(y.x) || not_finite<true>(y.y) ||
                                  not_finite<true>(y.z) || not_finite<true>(y.w));
            if (!row_stays(j, r, finite)) x = y = make_uint4(0, 0, 0, 0);
          }
          sts128(dst + r * 128 + (((2 * c) ^ (r & 7)) << 4), x);
          sts128(dst + r * 128 + (((2 * c + 1) ^ (r & 7)) << 4), y);
        }
        fence_async_smem();
      };
      if (!kFp8) {
        for (int j = 0; j < n_tiles; ++j) {
          // Every tile is waited for and let go, so that the barrier's phase is never lost.
          if (!ctx.wait_warp(BAR_V_FULL + (j & 1), (j >> 1) & 1)) break;
          if (!at_edge(j)) {
            if (lane == 0) mbar_arrive(ctx.bar(BAR_V_FREE + (j & 1)));
            continue;
          }
          clear_bad();
          const uint32_t vt = ctx.sbase + L::kV + (j & 1) * kTile16;
          for (int i = t; i < kTile * 4; i += 64) {
            // a lane's two chunks of its row, others' in other banks
            const int r = i >> 2;
            const uint32_t c0 = vt + r * 128 + 16 * ((2 * (i & 3) + r) & 7);
            const uint32_t c1 = vt + r * 128 + 16 * ((2 * (i & 3) + 1 + r) & 7);
            const uint4 x = lds128(c0), y = lds128(c1);
            const bool finite = !(not_finite<false>(x.x) || not_finite<false>(x.y) ||
                                  not_finite<false>(x.z) || not_finite<false>(x.w) ||
                                  not_finite<false>(y.x) || not_finite<false>(y.y) ||
                                  not_finite<false>(y.z) || not_finite<false>(y.w));
            if (!row_stays(j, r, finite)) {
              sts128(c0, make_uint4(0, 0, 0, 0));
              sts128(c1, make_uint4(0, 0, 0, 0));
            }
          }
          fence_async_smem();
          mbar_arrive(ctx.bar(BAR_SEEN + (edges & 1)));
          if (lane == 0) mbar_arrive(ctx.bar(BAR_V_FREE + (j & 1)));
          ++edges;
        }
      } else {
        // K of tile j+1 before V of tile j: Q K^T runs a tile ahead of P V
        auto convert_k = [&](int j) {
          const int s = j % kRaw;
          if (!ctx.wait_warp(BAR_RAW + s, (j / kRaw) & 1)) return false;
          if (j > 0 && !ctx.wait_warp(BAR_S_FULL, (j - 1) & 1)) return false;  // the one before is used
          convert(ctx.sbase + L::kRawK + s * kTile8, ctx.sbase + L::kK, false, j);
          mbar_arrive(ctx.bar(BAR_K_FULL));
          return true;
        };
        bool ok = n_tiles > 0 && convert_k(0);
        for (int j = 0; ok && j < n_tiles; ++j) {
          if (j + 1 < n_tiles && !(ok = convert_k(j + 1))) break;
          if (j > 0 && !(ok = ctx.wait_warp(BAR_PV, (j - 1) & 1))) break;  // V of the one before is used
          const bool look = at_edge(j);
          if (look) clear_bad();
          convert(ctx.sbase + L::kRawV + (j % kRaw) * kTile8, ctx.sbase + L::kV, look, j);
          mbar_arrive(ctx.bar(BAR_V_FULL));
          if (look) {
            mbar_arrive(ctx.bar(BAR_SEEN + (edges & 1)));
            ++edges;
          }
          mbar_arrive(ctx.bar(BAR_RAW_FREE + j % kRaw));
        }
      }
    }
  } else {
    // ------------------------------------------------------------------ softmax
    setmaxnreg_inc<kRegsSoftmax>();
    const int r = ht;  // row = TMEM lane
    const bool works = warp < active && !skip;
    float unit = 1.f;
    if (works)
      unit = store_query<kFp8>(a, smem, b, t0 + (r >> 3), idx0 + (r >> 3), g * kGroup + (r & 7), r);
    fence_async_smem();
    named_barrier(1, kThreads);  // the barriers and the tensor memory are there
    tc_fence_after_sync();
    const uint32_t tmem = *tmem_slot + half * kHalfCols;
    if (works) {
      const int t = t0 + (r >> 3);       // token
      const int idx = idx0 + (r >> 3);   // its index
      const uint32_t lane_off = static_cast<uint32_t>(warp * 32) << 16;
      const uint32_t tS = tmem + lane_off, tP = tS + kColP, tO = tS + kColO;
      {
        uint32_t z[32];
#pragma unroll
        for (int i = 0; i < 32; ++i) z[i] = 0u;
        tmem_st32(tO, z);
        tmem_st32(tO + 32, z);
        tmem_st_wait();
      }
      tc_fence_before_sync();
      mbar_arrive(ctx.bar(BAR_Q));

      float m = kNoMax, l = 0.f;
      const int first = a.window > 0 ? idx - a.window + 1 : 0;  // this row sees [first, idx]
      // the other half's barrier for this warp
      const uint32_t other_turn = ctx.bar(BAR_TURN + warp) +
                                  (half ? 0u - L::kHalfBytes : L::kHalfBytes);
      uint32_t edges = 0;  // tiles at the edge so far
      bool ok = true;
      uint32_t s_over = 0;
      for (int j = 0; j < n_tiles; ++j) {
        if (!(ok = ctx.wait_asked(s_over, BAR_S_FULL, j & 1))) break;
        tc_fence_after_sync();
        uint32_t sv[128];
        tmem_ld128_split(tS, sv);
        const int key0 = key_a + j * kTile;
        const bool edge = at_edge(j);
        const uint32_t turn_over = ctx.ask(BAR_TURN + warp, (half ? j : j - 1) & 1);
        const float4* pf = reinterpret_cast<const float4*>(smem + L::kPage + (j % kPageRing) * 128);
        if (!edge) {
          // S is in registers: the next product may overwrite it
          tc_fence_before_sync();
          __syncwarp();
          if (lane == 0) mbar_arrive(ctx.bar(BAR_S_FREE));
        }
        if (kFp8) {
          // scores in log2 units, with the page's value scale
#pragma unroll
          for (int p = 0; p < 8; ++p) {
            const float4 f = pf[p];
            const float c = f.x * unit;
            const uint64_t c2 = f2_pack(c, c), y2 = f2_pack(f.y, f.y);
#pragma unroll
            for (int e = 16 * p; e < 16 * p + 16; e += 2) {
              float x0, x1;
              f2_unpack(ffma2(f2_pack(__uint_as_float(sv[e]), __uint_as_float(sv[e + 1])), c2, y2),
                        x0, x1);
              sv[e] = __float_as_uint(x0);
              sv[e + 1] = __float_as_uint(x1);
            }
          }
        }
        if (edge) {
          const int c_hi = idx - key0, c_lo = first - key0;  // columns [c_lo, c_hi] are seen
#pragma unroll
          for (int i = 0; i < 128; ++i)
            if (i > c_hi || i < c_lo) sv[i] = __float_as_uint(-INFINITY);
        }
        float mx0 = kNoMax, mx1 = kNoMax, mx2 = kNoMax, mx3 = kNoMax;
#pragma unroll
        for (int i = 0; i < 128; i += 8) {
          mx0 = fmax3(mx0, __uint_as_float(sv[i]), __uint_as_float(sv[i + 1]));
          mx1 = fmax3(mx1, __uint_as_float(sv[i + 2]), __uint_as_float(sv[i + 3]));
          mx2 = fmax3(mx2, __uint_as_float(sv[i + 4]), __uint_as_float(sv[i + 5]));
          mx3 = fmax3(mx3, __uint_as_float(sv[i + 6]), __uint_as_float(sv[i + 7]));
        }
        float mx = fmaxf(fmaxf(mx0, mx1), fmaxf(mx2, mx3));
        if (!kFp8) mx = mx > kNoMax ? mx * kScaleLog2 : kNoMax;
        float alpha = 1.f;
        if (mx > m + kRescaleThreshold) {
          alpha = ex2_approx(m - mx);
          l *= alpha;
          m = mx;
        }
        // The halves' warps of a scheduler take turns: half 0 tile j, half 1 tile j, half 0
        // tile j+1, ...
        if ((j > 0 || half == 1) &&
            !(ok = ctx.wait_asked(turn_over, BAR_TURN + warp, (half ? j : j - 1) & 1)))
          break;
        // P and the sums' terms; a thread's 128 exponentials, packed in place
        const uint64_t c2 = f2_pack(kScaleLog2, kScaleLog2);
        const uint64_t nm2 = f2_pack(-m, -m);
        uint64_t acc0 = f2_pack(0.f, 0.f), acc1 = acc0;
        uint32_t pv_over = 0;
#pragma unroll
        for (int i = 0; i < 64; i += 2) {
          float x0, x1, x2, x3;
          const uint64_t u = f2_pack(__uint_as_float(sv[2 * i]), __uint_as_float(sv[2 * i + 1]));
          const uint64_t v = f2_pack(__uint_as_float(sv[2 * i + 2]), __uint_as_float(sv[2 * i + 3]));
          f2_unpack(kFp8 ? fadd2(u, nm2) : ffma2(u, c2, nm2), x0, x1);
          f2_unpack(kFp8 ? fadd2(v, nm2) : ffma2(v, c2, nm2), x2, x3);
          const float p0 = ex2_approx(x0), p1 = ex2_approx(x1);
          const float p2 = ex2_approx(x2), p3 = ex2_approx(x3);
          acc0 = fadd2(acc0, f2_pack(p0, p1));
          acc1 = fadd2(acc1, f2_pack(p2, p3));
          sv[i] = kFp8 ? pack_f16x2(p0, p1) : pack_bf16x2(p0, p1);
          sv[i + 1] = kFp8 ? pack_f16x2(p2, p3) : pack_bf16x2(p2, p3);
          if (i == kAskPv) pv_over = ctx.ask(BAR_PV, (j - 1) & 1);
          if (i == kTurnHandOff) {
            __syncwarp();
            if (lane == 0) mbar_arrive(other_turn);
          }
          if (kFp8 && i % 8 == 6) {  // the end of a page's 16 columns
            float s0, s1, s2, s3;
            f2_unpack(acc0, s0, s1);
            f2_unpack(acc1, s2, s3);
            l = fmaf((s0 + s1) + (s2 + s3), pf[i / 8].z, l);
            acc0 = acc1 = f2_pack(0.f, 0.f);
          }
        }
        if (!kFp8) {
          float s0, s1, s2, s3;
          f2_unpack(acc0, s0, s1);
          f2_unpack(acc1, s2, s3);
          l += (s0 + s1) + (s2 + s3);
        }
        // P and O are this warpgroup's once the previous tile's P V is done
        if (j > 0 && !(ok = ctx.wait_asked(pv_over, BAR_PV, (j - 1) & 1))) break;
        tc_fence_after_sync();
        s_over = ctx.ask(BAR_S_FULL, (j + 1) & 1);
        {
          uint32_t pw[64];
#pragma unroll
          for (int i = 0; i < 64; ++i) pw[i] = sv[i];
          tmem_st64(tP, pw);
        }
        if (j > 0 && __any_sync(0xffffffffu, alpha != 1.f)) {
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            uint32_t ov[32];
            tmem_ld32(tO + 32 * half, ov);
#pragma unroll
            for (int i = 0; i < 32; ++i) ov[i] = __float_as_uint(__uint_as_float(ov[i]) * alpha);
            tmem_st32(tO + 32 * half, ov);
          }
        }
        tmem_st_wait();
        if (edge) {
          // value rows that were taken out of the tile
          if (!(ok = ctx.wait_warp(BAR_SEEN + (edges & 1), (edges >> 1) & 1))) break;
          const uint32_t* bad = reinterpret_cast<const uint32_t*>(smem + L::kBad) + 8 * (edges & 1);
          ++edges;
          for (int word = 0; word < 4; ++word) {
            for (uint32_t bits = bad[word] | bad[4 + word]; bits; bits &= bits - 1) {
              const int k = 32 * word + __ffs(bits) - 1;
              const int key = key0 + k;
              float s = tmem_ld1(tS + k);
              s = kFp8 ? fmaf(s, pf[k >> 4].x * unit, pf[k >> 4].y - m) : fmaf(s, kScaleLog2, -m);
              const bool see = key >= first && key <= idx;
              const float p = see ? ex2_approx(s) : 0.f;
              const int page = __ldg(table + (key >> page_log2));
              const int64_t at = page * a.cache.page_stride +
                                 (key & ((1 << page_log2) - 1)) * a.cache.token_stride +
                                 g * a.cache.head_stride;
              for (int half = 0; half < 2; ++half) {
                uint32_t ov[32];
                tmem_ld32(tO + 32 * half, ov);
#pragma unroll
                for (int d = 0; d < 32; d += 2) {
                  uint32_t w;
                  float v0, v1;
                  if (kFp8) {
                    uint32_t unused;
                    e4m3x4_to_f16(*reinterpret_cast<const uint16_t*>(a.cache.v + at + 32 * half + d),
                                  w, unused);
                    asm("{\n\t.reg .b16 x, y;\n\tmov.b32 {x, y}, %2;\n\tcvt.f32.f16 %0, x;\n\t"
                        "cvt.f32.f16 %1, y;\n\t}"
                        : "=f"(v0), "=f"(v1)
                        : "r"(w));
                  } else {
                    w = *reinterpret_cast<const uint32_t*>(a.cache.v + 2 * (at + 32 * half + d));
                    v0 = bf16lo_to_f32(w);
                    v1 = bf16hi_to_f32(w);
                  }
                  if (see) {
                    ov[d] = __float_as_uint(fmaf(p, v0, __uint_as_float(ov[d])));
                    ov[d + 1] = __float_as_uint(fmaf(p, v1, __uint_as_float(ov[d + 1])));
                  }
                }
                tmem_st32(tO + 32 * half, ov);
              }
              tmem_st_wait();
            }
          }
          tc_fence_before_sync();
          __syncwarp();
          if (lane == 0) mbar_arrive(ctx.bar(BAR_S_FREE));
        }
        tc_fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(ctx.bar(BAR_P_FULL));
      }
      // ---- the row's sums: its output, or a part
      if (ok && n_tiles > 0) ok = ctx.wait_warp(BAR_PV, (n_tiles - 1) & 1);
      if (kFp8 && ok && *far) {
        const int tokens = min(kNT, a.n - t0);
#pragma unroll 1
        for (int i = 2 * warp + (lane >> 4); i < tokens * kGroup; i += 2 * active)
          plain_row(a, b, t0 + i / kGroup, idx0 + i / kGroup, g * kGroup + i % kGroup, key_a,
                    key_a + n_tiles * kTile, chunks,
                    (static_cast<int64_t>(part) * kNumKvHeads + g) * (kNT * kGroup) + i);
      } else if (ok) {
        tc_fence_after_sync();
        const bool write = t < a.n;
        float scale = 1.f;
        const float grow = kFp8 ? paged_power(*unit_of) : 1.f;
        if (chunks == 1) {
          const float sink = __ldg(a.sinks + g * kGroup + (r & 7)) * kLog2e;
          const float Mf = fmaxf(sink, m);
          const float f = ex2_approx(m - Mf);
          scale = m > kNoMax ? f / fmaf(f, l, ex2_approx(sink - Mf)) : 0.f;
        }
        const int64_t pr = (static_cast<int64_t>(part) * kNumKvHeads + g) * (kNT * kGroup) + r;
        const int64_t orow = (static_cast<int64_t>(b) * a.n + t) * kNumHeads + g * kGroup + (r & 7);
        uint32_t ov[2][32];
        tmem_ld32(tO, ov[0]);
        tmem_ld32(tO + 32, ov[1]);
        if (write && chunks == 1) {
#pragma unroll
          for (int i = 0; i < 64; i += 8) {
            uint32_t w[4];
#pragma unroll
            for (int e = 0; e < 4; ++e)
              w[e] = pack_bf16x2(__uint_as_float(ov[i / 32][i % 32 + 2 * e]) * scale * grow,
                                 __uint_as_float(ov[i / 32][i % 32 + 2 * e + 1]) * scale * grow);
            *reinterpret_cast<uint4*>(a.out + orow * kHeadDim + i) =
                make_uint4(w[0], w[1], w[2], w[3]);
          }
        } else if (write) {
          const float2 f = kFp8 ? to_part(&m, &l, *unit_of) : make_float2(1.f, 1.f);
#pragma unroll
          for (int i = 0; i < 64; i += 4) {
            float o[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              o[e] = __uint_as_float(ov[i / 32][i % 32 + e]);
              if (kFp8) o[e] = o[e] * f.x * f.y;
            }
            *reinterpret_cast<float4*>(a.part_o + pr * kHeadDim + i) =
                make_float4(o[0], o[1], o[2], o[3]);
          }
          a.part_ml[pr] = make_float2(m, l);
        }
      }
    }
  }

  tc_fence_before_sync();
  __syncthreads();
  if (half == 0 && warp == 5) {
    tc_fence_after_sync();
    tmem_dealloc(*tmem_slot, kTmemCols);
  }
}

template <bool kFp8>
cudaError_t launch(const PagedMaps& maps, const PagedAttentionArgs& a, cudaStream_t stream) {
  using L = Smem<kFp8>;
  static std::atomic<uint64_t> prepared{0};  // devices whose kernel has its shared memory
  cudaError_t e = allow_shared(reinterpret_cast<const void*>(paged_many_kernel<kFp8>), L::kBytes,
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
  cfg.gridDim = dim3(static_cast<unsigned>(chunks * kNumKvHeads / 2));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = L::kBytes;
  e = cudaLaunchKernelEx(&cfg, paged_many_kernel<kFp8>, maps, a);
  if (e != cudaSuccess || a.none_cut) return e;
  return launch_paged_combine(a, kNT, stream);
}

}  // namespace

cudaError_t launch_paged_attention_many(const PagedMaps& maps, const PagedAttentionArgs& a,
                                        cudaStream_t stream) {
  return a.cache.fp8 ? launch<true>(maps, a, stream) : launch<false>(maps, a, stream);
}

}  // namespace gqa
