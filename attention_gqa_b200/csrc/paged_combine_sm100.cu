// The second kernel of attention over a paged cache: joins the chunks of rows that
// were cut (a log-sum-exp merge with the sink counted once), and the sizes that both
// attention kernels plan with.
#include "paged_common.cuh"

namespace gqa {
namespace {

// Joins the chunks of the rows that have several, with the sink, normalises and
// rounds. A CTA takes kHeads heads of one token. With one head, each of 16 warps
// takes every sixteenth chunk and the warps join at the end (few rows, which may
// have many chunks); with eight, a warp takes a head (many rows).
template <int NT, int kHeads>
__global__ void __launch_bounds__(kHeads == 1 ? 512 : 256) paged_combine_kernel(const PagedAttentionArgs a) {
  griddep_launch_dependents();
  griddep_wait();
  constexpr int kSplit = kHeads == 1 ? 16 : 1;  // warps per head
  __shared__ float2 part[kSplit][32];
  __shared__ float2 part_ml[kSplit];
  const int warp = static_cast<int>(threadIdx.x >> 5), lane = static_cast<int>(threadIdx.x & 31);
  const int row = static_cast<int>(blockIdx.x);
  const int r = static_cast<int>(blockIdx.y) * kHeads + warp / kSplit;  // token of the row, head
  const int tk = r / kNumHeads, h = r % kNumHeads;
  const int2 meta = a.meta[row];
  const int b = row / a.groups, t = (row - b * a.groups) * NT + tk;
  if (meta.y == 1 || t >= a.n || (*reinterpret_cast<volatile int*>(a.err) & kErrTimeout)) return;
  const int64_t stride = kNumKvHeads * NT * kGroup;
  const int64_t first = meta.x * stride + (h / kGroup) * (NT * kGroup) + tk * kGroup + h % kGroup;
  float M = kNoMax, sum = 0.f, o0 = 0.f, o1 = 0.f;
  constexpr int kBatch = 8;
  for (int s0 = warp % kSplit; s0 < meta.y; s0 += kBatch * kSplit) {
    float2 ml[kBatch], v[kBatch];
#pragma unroll
    for (int j = 0; j < kBatch; ++j) {
      const int s = s0 + j * kSplit;
      ml[j] = make_float2(kNoMax, 0.f);
      v[j] = make_float2(0.f, 0.f);
      if (s < meta.y) {
        ml[j] = a.part_ml[first + s * stride];
        v[j] = *reinterpret_cast<const float2*>(a.part_o + (first + s * stride) * kHeadDim +
                                                2 * lane);
      }
    }
    float top = M;
#pragma unroll
    for (int j = 0; j < kBatch; ++j) top = fmaxf(top, ml[j].x);
    const float f = ex2_approx(M - top);
    M = top;
    sum *= f;
    o0 *= f;
    o1 *= f;
#pragma unroll
    for (int j = 0; j < kBatch; ++j) {
      const float fj = ex2_approx(ml[j].x - top);
      sum = fmaf(fj, ml[j].y, sum);
      o0 = fmaf(fj, v[j].x, o0);
      o1 = fmaf(fj, v[j].y, o1);
    }
  }
  const float sink = __ldg(a.sinks + h) * kLog2e;
  float Mf = fmaxf(sink, M), den;
  if (kSplit > 1) {
    part[warp][lane] = make_float2(o0, o1);
    if (lane == 0) part_ml[warp] = make_float2(M, sum);
    __syncthreads();
    if (warp > 0) return;
    Mf = sink;
    for (int w = 0; w < kSplit; ++w) Mf = fmaxf(Mf, part_ml[w].x);
    den = ex2_approx(sink - Mf);
    o0 = o1 = 0.f;
    for (int w = 0; w < kSplit; ++w) {
      const float f = ex2_approx(part_ml[w].x - Mf);
      den = fmaf(f, part_ml[w].y, den);
      o0 = fmaf(f, part[w][lane].x, o0);
      o1 = fmaf(f, part[w][lane].y, o1);
    }
  } else {
    const float f = ex2_approx(M - Mf);
    den = fmaf(f, sum, ex2_approx(sink - Mf));
    o0 *= f;
    o1 *= f;
  }
  const float inv = den > 0.f ? 1.f / den : 0.f;
  reinterpret_cast<uint32_t*>(a.out + ((static_cast<int64_t>(b) * a.n + t) * kNumHeads + h) *
                                          kHeadDim)[lane] = pack_bf16x2(o0 * inv, o1 * inv);
}

template <int NT>
cudaError_t launch(cudaLaunchConfig_t& cfg, const PagedAttentionArgs& a) {
  // the first form while its CTAs, one per output row, are few
  const bool few = static_cast<int64_t>(a.rows) * NT <= 16;
  cfg.blockDim = dim3(few ? 512 : 256);
  cfg.gridDim = dim3(static_cast<unsigned>(a.rows), NT * (few ? kNumHeads : kNumKvHeads));
  return few ? cudaLaunchKernelEx(&cfg, paged_combine_kernel<NT, 1>, a)
             : cudaLaunchKernelEx(&cfg, paged_combine_kernel<NT, 8>, a);
}

}  // namespace

cudaError_t launch_paged_combine(const PagedAttentionArgs& a, int row_tokens, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cfg.stream = stream;
  switch (row_tokens) {
    case 1: return launch<1>(cfg, a);
    case 2: return launch<2>(cfg, a);
    default: return launch<kPagedManyTokens>(cfg, a);
  }
}

int paged_row_tokens(int n) { return n <= 2 ? n : kPagedManyTokens; }

// Chunks that the GPU holds at a time: eight CTAs of the kernel for few tokens, one per kv
// head, are a chunk, four of the other.
static int paged_wave(int row_tokens, bool fp8) {
  const int per_sm = row_tokens == 1 ? (fp8 ? 4 : 3) : row_tokens == 2 ? 3 : 2;
  return 148 * per_sm / kNumKvHeads;
}

// Of many rows: chunks aimed for, at most.
static int paged_target(int row_tokens, bool fp8) {
  return row_tokens == 1 ? (fp8 ? 111 : 148) : row_tokens == 2 ? 111 : 37;
}

// A chunk costs about 6 us before its first tile, as much as many tiles, so rows that leave
// room for it are cut to exactly one wave (1 x 131072 e4m3: 32.7 us against 42.7 with 222
// chunks; 8 x 32768 e4m3: 57 against 64; 32 ragged rows of 4096 bf16: 32.9 against 38).
// More rows make uneven chunks, which are better dealt out in one and a half to three
// waves (64 ragged rows of 8192 e4m3: 62.5 us at 111 chunks, 67.8 at 74, 68.7 at 222; 64
// full rows bf16: 172 us at 148, 177 at 74). Many tokens: a wave, and less by half a chunk
// a row, of which the last is half empty on average.
void paged_plan(PagedAttentionArgs* a) {
  const int nt = paged_row_tokens(a->n);
  const int wave = paged_wave(nt, a->cache.fp8);
  a->one_wave = 4 * static_cast<int64_t>(a->rows) <= 3 * wave;
  a->target = a->one_wave ? wave : paged_target(nt, a->cache.fp8);
  if (nt == kPagedManyTokens && !a->one_wave && a->rows < wave) a->target -= a->rows / 2;
}

int paged_most_tiles(int nt, int tile, int max_len, int window) {
  // a row of nt tokens sees window + nt - 1 keys, from anywhere in a tile
  return paged_row_tiles(0, window > 0 && window + nt + tile < max_len ? window + nt + tile : max_len,
                         tile);
}

size_t paged_workspace_bytes(int64_t rows, int n, int max_len, int window, size_t off[3]) {
  const int nt = paged_row_tokens(n);
  // (a wave is fewer chunks, and so are those of e4m3 pages)
  const size_t parts = static_cast<size_t>(paged_max_parts(paged_target(nt, false))) * kNumKvHeads *
                       nt * kGroup;
  off[0] = 0;
  off[1] = parts * kHeadDim * sizeof(float);
  off[2] = off[1] + parts * sizeof(float2);
  // (the kernel for few tokens takes longer tiles of e4m3 pages, and cuts them less)
  const int most = paged_most_tiles(nt, nt <= 2 ? kPagedTile : kPagedTileN, max_len, window);
  if (most <= kPagedWhole) return 0;
  return off[2] + ((static_cast<size_t>(rows) * sizeof(int2) + 15) & ~static_cast<size_t>(15));
}

}  // namespace gqa
