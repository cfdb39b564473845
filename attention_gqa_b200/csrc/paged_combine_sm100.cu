// The second kernel of attention over a paged cache: joins the chunks of rows that
// were cut (a log-sum-exp merge with the sink counted once), and the sizes that both
// attention kernels plan with.
#include "paged_common.cuh"

namespace gqa {
namespace {

constexpr int kWarps = 8;
constexpr int kThreads = 32 * kWarps;

// Lanes of a head, and heads of a CTA.
template <int kSplit>
struct Form {
  static constexpr int kLanes = kSplit == 1 ? 8 : 32;
  static constexpr int kHeads = kWarps / kSplit * (32 / kLanes);
};

// Joins the chunks of the rows that have several, with the sink, normalises and rounds.
// kSplit > 1 (few rows, of many chunks): so many warps take a head of a token, each every
// kSplit-th chunk, and join at the end. kSplit = 1: a warp takes four heads. Most rows of a
// call may have one chunk and nothing to join, so that is what a CTA looks at first (512
// tokens on 4096, none cut: 79.2 us with both kernels against 83.4 with a warp per head).
// nt: tokens of a row.
template <int kSplit>
__global__ void __launch_bounds__(kThreads, 4)
    paged_combine_kernel(const PagedAttentionArgs a, int nt) {
  using F = Form<kSplit>;
  constexpr int kPer = kHeadDim / F::kLanes;  // elements of a lane
  griddep_wait();
  const int row = static_cast<int>(blockIdx.x);
  constexpr int kCtas = kNumHeads / F::kHeads;  // of a token
  const int tk = static_cast<int>(blockIdx.y) / kCtas;
  const int b = row / a.groups, t = (row - b * a.groups) * nt + tk;
  const int warp = static_cast<int>(threadIdx.x >> 5), lane = static_cast<int>(threadIdx.x & 31);
  const int h = static_cast<int>(blockIdx.y) % kCtas * F::kHeads +
                (warp / kSplit) * (32 / F::kLanes) + lane / F::kLanes;
  const int d0 = lane % F::kLanes * kPer;
  const int2 meta = a.meta[row];
  if (t >= a.n || meta.y == 1 || (*reinterpret_cast<volatile int*>(a.err) & kErrTimeout)) return;
  // (32 bits: the parts are few, whatever the rows)
  const int stride = kNumKvHeads * nt * kGroup;
  const int first = meta.x * stride + (h / kGroup) * (nt * kGroup) + tk * kGroup + h % kGroup;
  float M = kNoMax, sum = 0.f, o[kPer];
#pragma unroll
  for (int e = 0; e < kPer; ++e) o[e] = 0.f;
  constexpr int kBatch = kSplit == 1 ? 4 : 8;  // loads in flight
#pragma unroll 1
  for (int s0 = warp % kSplit; s0 < meta.y; s0 += kBatch * kSplit) {
    float2 ml[kBatch], v[kBatch][kPer / 2];
#pragma unroll
    for (int j = 0; j < kBatch; ++j) {
      const int s = s0 + j * kSplit;
      ml[j] = make_float2(kNoMax, 0.f);
#pragma unroll
      for (int e = 0; e < kPer / 2; ++e) v[j][e] = make_float2(0.f, 0.f);
      if (s < meta.y) {
        const int at = first + s * stride;
        ml[j] = a.part_ml[at];
        if constexpr (kPer == 2) {
          v[j][0] = *reinterpret_cast<const float2*>(a.part_o + at * kHeadDim + d0);
        } else {
#pragma unroll
          for (int e = 0; e < kPer / 2; e += 2) {
            const float4 w = *reinterpret_cast<const float4*>(a.part_o + at * kHeadDim + d0 + 2 * e);
            v[j][e] = make_float2(w.x, w.y);
            v[j][e + 1] = make_float2(w.z, w.w);
          }
        }
      }
    }
    float top = M;
#pragma unroll
    for (int j = 0; j < kBatch; ++j) top = fmaxf(top, ml[j].x);
    const float f = ex2_approx(M - top);
    M = top;
    sum *= f;
#pragma unroll
    for (int e = 0; e < kPer; ++e) o[e] *= f;
#pragma unroll
    for (int j = 0; j < kBatch; ++j) {
      const float fj = ex2_approx(ml[j].x - top);
      sum = fmaf(fj, ml[j].y, sum);
#pragma unroll
      for (int e = 0; e < kPer; e += 2) {
        o[e] = fmaf(fj, v[j][e / 2].x, o[e]);
        o[e + 1] = fmaf(fj, v[j][e / 2].y, o[e + 1]);
      }
    }
  }
  // Not earlier: a next call's CTAs would take their places while these hold registers, and
  // no longer fit one wave.
  griddep_launch_dependents();
  const float sink = __ldg(a.sinks + h) * kLog2e;
  float Mf = fmaxf(sink, M), den;
  if constexpr (kSplit > 1) {
    __shared__ float2 part[kWarps][32];
    __shared__ float2 part_ml[kWarps];
    part[warp][lane] = make_float2(o[0], o[1]);
    if (lane == 0) part_ml[warp] = make_float2(M, sum);
    __syncthreads();
    if (warp % kSplit != 0) return;
    Mf = sink;
#pragma unroll 1
    for (int w = 0; w < kSplit; ++w) Mf = fmaxf(Mf, part_ml[warp + w].x);
    den = ex2_approx(sink - Mf);
    o[0] = o[1] = 0.f;
#pragma unroll 1
    for (int w = 0; w < kSplit; ++w) {
      const float f = ex2_approx(part_ml[warp + w].x - Mf);
      den = fmaf(f, part_ml[warp + w].y, den);
      o[0] = fmaf(f, part[warp + w][lane].x, o[0]);
      o[1] = fmaf(f, part[warp + w][lane].y, o[1]);
    }
  } else {
    const float f = ex2_approx(M - Mf);
    den = fmaf(f, sum, ex2_approx(sink - Mf));
#pragma unroll
    for (int e = 0; e < kPer; ++e) o[e] *= f;
  }
  const float inv = den > 0.f ? 1.f / den : 0.f;
  uint32_t w[kPer / 2];
#pragma unroll
  for (int e = 0; e < kPer; e += 2) w[e / 2] = pack_bf16x2(o[e] * inv, o[e + 1] * inv);
  uint32_t* out = reinterpret_cast<uint32_t*>(
      a.out + ((static_cast<int64_t>(b) * a.n + t) * kNumHeads + h) * kHeadDim + d0);
  if constexpr (kPer == 2) {
    *out = w[0];
  } else {
    *reinterpret_cast<uint4*>(out) = make_uint4(w[0], w[1], w[2], w[3]);
  }
}

template <int kSplit>
cudaError_t launch(cudaLaunchConfig_t& cfg, const PagedAttentionArgs& a, int nt) {
  using F = Form<kSplit>;
  cfg.blockDim = dim3(kThreads);
  cfg.gridDim = dim3(static_cast<unsigned>(a.rows), nt * kNumHeads / F::kHeads);
  return cudaLaunchKernelEx(&cfg, paged_combine_kernel<kSplit>, a, nt);
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
  // by the chunks that a row has on average; and eight warps while they are few (one row of
  // 131072, 74 chunks: 33 us with eight or sixteen warps a head, 43 when one read 222 chunks
  // in turn; one row of 16 tokens on 32768: 33.6 us with four, 38 with sixteen)
  const int chunks = a.target / a.rows;
  if (chunks >= 16 && a.rows * row_tokens <= 8) return launch<8>(cfg, a, row_tokens);
  return chunks >= 8 ? launch<4>(cfg, a, row_tokens) : launch<1>(cfg, a, row_tokens);
}

int paged_row_tokens(int n) { return n <= 2 ? n : kPagedManyTokens; }

static int paged_most_tiles(int nt, int tile, int max_len, int window) {
  // a row of nt tokens sees window + nt - 1 keys, from anywhere in a tile
  return paged_row_tiles(0, window > 0 && window + nt + tile < max_len ? window + nt + tile : max_len,
                         tile);
}

// A chunk costs about 6 us before its first tile, as much as many tiles, so rows that leave
// room for it are cut to exactly one wave (1 x 131072 e4m3: 33 us against 43 with 222
// chunks; 8 x 32768 e4m3: 55 against 64; 32 ragged rows of 4096 bf16: 31 against 36).
// More rows make uneven chunks, which are better dealt out in a wave and a half (64 ragged
// rows of 8192 e4m3: 61 us at 111 chunks, 67 at 74, 70 at 222; 64 full rows bf16: 167 us
// at 111, 166 at 74, 174 at 222). With many tokens a chunk has its SM alone and its time
// is known better, so the device estimates whether whole rows end first (36 full rows of
// 8192 e4m3, five tokens each: 139 us whole, 152 cut; 36 ragged ones: 124 and 103; eight
// pieces of 40 on 32768: 555 us whole, 397 cut).
void paged_plan(PagedAttentionArgs* a, int num_sms) {
  const int nt = paged_row_tokens(a->n);
  const bool many = nt == kPagedManyTokens;
  a->wave = paged_wave(nt, num_sms);
  a->most = paged_most_tiles(nt, !many && !a->cache.fp8 ? kPagedTile : kPagedTileN, a->max_len,
                             a->window);
  a->none_cut = paged_none_cut(a->rows, a->most);
  a->one_wave = a->rows <= (many ? a->wave / 2 : 3 * a->wave / 4);
  a->target = a->one_wave ? a->wave : paged_target(nt);
}

size_t paged_workspace_bytes(int64_t rows, int n, int max_len, int window, size_t off[3]) {
  const int nt = paged_row_tokens(n);
  // (a wave is no more chunks)
  const size_t parts = static_cast<size_t>(paged_max_parts(paged_target(nt))) * kNumKvHeads *
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
