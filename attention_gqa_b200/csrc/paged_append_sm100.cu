// Appending keys and values to a paged cache for sm_100a, keys rotated on the way.
//
// Token t of a sequence's `count` new ones sits at index i = len - count + t, in
// page table[b][i / P] at slot i % P. bf16 pages take the rotated key (fp32
// arithmetic from the fp64-built table, one rounding, as rope_rows_kernel does
// it) and the value as given. e4m3 pages hold x / s with one scale s per page
// and head, a power of two so that a later, larger scale moves the codes that
// are there without rounding them again (but for those that get subnormal):
//   s = max(s of the page's earlier tokens, least 2^e with max |x| <= 448 * 2^e).
// Infinities saturate and NaN stays; neither decides the scale. A rotation may pass fp32's
// range (bf16's largest, times sqrt 2 and YaRN's factor); what it gives is finite all the same.
//
// Both kernels have HBM's floor: 256 bytes read per token and kv head, 256 (bf16) or 128
// (e4m3) written. Measured on a B200 for 4 x 16384 tokens: bf16 43.5 us, 6.2 TB/s of that;
// e4m3 51.5 us, 3.9 TB/s, whose CTAs wait in turn for their tokens and for their largest value
// (64 registers a thread allow 32 warps per SM, and 61 % of the issue slots are used). One
// token of 64 sequences: 1.7 and 2.7 us on the device, less than a launch.
#include <cfloat>
#include <cmath>

#include "internal.h"
#include "paged.h"
#include "sm100_ptx.cuh"

namespace gqa {
namespace {

// (cos, sin) of pairs 8c .. 8c+7 of a table row.
struct Turn {
  float c[8], s[8];
  __device__ __forceinline__ void load(const float2* row, int chunk) {
    const float4* t4 = reinterpret_cast<const float4*>(row + 8 * chunk);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float4 t = __ldg(t4 + i);
      c[2 * i] = t.x;
      s[2 * i] = t.y;
      c[2 * i + 1] = t.z;
      s[2 * i + 1] = t.w;
    }
  }
};

// Elements 8c .. 8c+7 (lo) and 8c+32 .. 8c+39 (hi) of a head, as fp32.
struct Halves {
  float lo[8], hi[8];
  __device__ __forceinline__ void unpack(const uint4& a, const uint4& h) {
    const uint32_t aw[4] = {a.x, a.y, a.z, a.w}, hw[4] = {h.x, h.y, h.z, h.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      lo[2 * e] = bf16lo_to_f32(aw[e]);
      lo[2 * e + 1] = bf16hi_to_f32(aw[e]);
      hi[2 * e] = bf16lo_to_f32(hw[e]);
      hi[2 * e + 1] = bf16hi_to_f32(hw[e]);
    }
  }
  // lo cos - hi sin, hi cos + lo sin; as the rotation of the other entry points rounds them
  __device__ __forceinline__ void turn(const Turn& t) {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float a = lo[e], h = hi[e];
      lo[e] = fmaf(a, t.c[e], -h * t.s[e]);
      hi[e] = fmaf(h, t.c[e], a * t.s[e]);
    }
  }
  // The same with each result's error an ulp at most (the product's rounding error is
  // added back): codes are fp32 values rounded once more, so an error of the sum
  // shows wherever a value lies at a border between two codes.
  __device__ __forceinline__ void turn_exactly(const Turn& t) {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float a = lo[e], h = hi[e];
      const float hs = h * t.s[e], as = a * t.s[e];
      lo[e] = fmaf(a, t.c[e], -hs) + fmaf(-h, t.s[e], hs);
      hi[e] = fmaf(h, t.c[e], as) + fmaf(a, t.s[e], -as);
    }
  }
};

__device__ __forceinline__ uint4 pack8(const float (&x)[8]) {
  return make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]),
                    pack_bf16x2(x[6], x[7]));
}

// Table row of a token's position; one outside the table is reported and clamped.
__device__ __forceinline__ const float2* table_row(const PagedAppendArgs& a, int b, int t) {
  int p = __ldg(a.pos + static_cast<int64_t>(b) * a.n + t);
  if (p < 0 || p >= kMaxPosition) {
    atomicOr(a.err, kErrPosition);
    p = p < 0 ? 0 : kMaxPosition - 1;
  }
  return a.rope + static_cast<int64_t>(p) * kRopePairs;
}

// Where a sequence's new tokens start and how many there are; a call that does
// not fit its sequence is reported and appends nothing to it. Nor does one behind a
// kernel whose waits timed out: its tokens may be anything, and a page's scale would
// keep what they were.
__device__ __forceinline__ bool new_tokens(const PagedAppendArgs& a, int b, int* start,
                                           int* count) {
  const int err = *a.err;  // (through L1: read past it by every warp, it costs prompts 7 %)
  const int len = __ldg(a.len + b);
  const int c = a.count ? __ldg(a.count + b) : a.n;
  if (err & kErrTimeout) return false;
  if (!paged_append_ok(len, c, a.n, a.max_len)) {
    atomicOr(a.err, kErrLength);
    return false;
  }
  *start = len - c;
  *count = c;
  return true;
}

// One warp per token, four lanes per kv head: lane c of a head takes the 16-byte
// chunks c and c+4, which the rotation pairs, of its key and of its value.
__global__ void __launch_bounds__(256) append_bf16_kernel(const PagedAppendArgs a) {
  griddep_launch_dependents();
  griddep_wait();  // lengths, tokens and pages may come from the kernel before
  const int b = static_cast<int>(blockIdx.y);
  const int t = static_cast<int>(blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5));
  const int lane = static_cast<int>(threadIdx.x & 31);
  const int head = lane >> 2, c = lane & 3;
  int start, count;
  if (t >= a.n || !new_tokens(a, b, &start, &count) || t >= count) return;
  const PagedCache& pc = a.cache;
  const int i = start + t;
  const int page = __ldg(a.table + static_cast<int64_t>(b) * a.max_pages + (i >> pc.page_log2));
  const uint4* k4 = reinterpret_cast<const uint4*>(a.k + b * a.k_batch + t * a.k_token +
                                                   head * kHeadDim);
  const uint4* v4 = reinterpret_cast<const uint4*>(a.v + b * a.v_batch + t * a.v_token +
                                                   head * kHeadDim);
  const uint4 klo = __ldg(k4 + c), khi = __ldg(k4 + c + 4);
  const uint4 vlo = __ldg(v4 + c), vhi = __ldg(v4 + c + 4);
  Turn turn;
  turn.load(table_row(a, b, t), c);
  if (!paged_page_ok(page, pc.num_pages)) {
    if (lane == 0) atomicOr(a.err, kErrPage);
    return;
  }
  Halves x;
  x.unpack(klo, khi);
  x.turn(turn);
  const int64_t at = page * pc.page_stride +
                     (i & ((1 << pc.page_log2) - 1)) * pc.token_stride + head * pc.head_stride;
  uint4* ko = reinterpret_cast<uint4*>(pc.k + 2 * at);
  uint4* vo = reinterpret_cast<uint4*>(pc.v + 2 * at);
  ko[c] = pack8(x.lo);
  ko[c + 4] = pack8(x.hi);
  vo[c] = vlo;
  vo[c + 4] = vhi;
}

// Two fp32 values to two e4m3 codes (round to nearest even, saturating; NaN stays).
__device__ __forceinline__ uint32_t pack_e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}

__device__ __forceinline__ uint2 pack_e4m3x8(const float (&x)[8], float f) {
  return make_uint2(pack_e4m3x2(x[0] * f, x[1] * f) | pack_e4m3x2(x[2] * f, x[3] * f) << 16,
                    pack_e4m3x2(x[4] * f, x[5] * f) | pack_e4m3x2(x[6] * f, x[7] * f) << 16);
}

// The two values of two codes.
__device__ __forceinline__ float2 unpack_e4m3x2(uint32_t codes) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(static_cast<uint16_t>(codes)));
  float lo, hi;
  asm("{\n\t.reg .b16 l, u;\n\tmov.b32 {l, u}, %2;\n\tcvt.f32.f16 %0, l;\n\tcvt.f32.f16 %1, u;\n\t}"
      : "=f"(lo), "=f"(hi)
      : "r"(h));
  return make_float2(lo, hi);
}

__device__ __forceinline__ uint32_t move_e4m3x4(uint32_t codes, float f) {
  const float2 a = unpack_e4m3x2(codes & 0xFFFFu), b = unpack_e4m3x2(codes >> 16);
  return pack_e4m3x2(a.x * f, a.y * f) | pack_e4m3x2(b.x * f, b.y * f) << 16;
}

// The largest |value|, NaN aside; infinite if there is an infinity, or a sum beyond fp32's range.
__device__ __forceinline__ float largest(const Halves& x, float top) {
#pragma unroll
  for (int e = 0; e < 8; ++e) top = fmax3(top, fabsf(x.lo[e]), fabsf(x.hi[e]));
  return top;
}

constexpr int kAppendWarps = 16;  // most warps of a CTA
// Below this no product or sum of a rotation overflows fp32, nor does an infinity hide: one
// element of a pair at least is infinite if an input was.
constexpr float kWide = 0x1p127f;

// Eight CTAs per page that a sequence's new tokens touch, for two heads of its keys or of its
// values each: the scale needs the largest of all the page's new values, and the smaller
// the CTA that waits for them, the better its waits pass under others' work. Eight lanes
// take a token, four a head as above (256 bytes in a row); a warp's tokens, at most kTokens to
// a lane, are read once and kept, for the largest value of each head over the CTA and
// then for the codes. For 4 x 16384 tokens in pages of 16, 32, 64 and 128: 51, 52, 51 and 56
// us; with four heads in a CTA 51, 50, 54 and 61; with eight 81, 60, 57 and 65; with keys and
// values in one, 63 to 70 (64); a warp per (page, head) that reads twice, 90 (64). For 7 x
// 333 in pages of 128: 6.6 us; with four heads 8.3, with eight 13.9.
template <int kTokens>
__global__ void __launch_bounds__(32 * kAppendWarps, 2)
    append_e4m3_kernel(const PagedAppendArgs a) {
  griddep_launch_dependents();
  griddep_wait();
  __shared__ float tops[kAppendWarps][2];  // by warp and head
  const int b = static_cast<int>(blockIdx.y);
  const int warp = static_cast<int>(threadIdx.x >> 5), lane = static_cast<int>(threadIdx.x & 31);
  const int warps = static_cast<int>(blockDim.x >> 5);
  const int sub = lane >> 3;  // which token of the warp's four
  const int local = (lane >> 2) & 1, c = lane & 3;
  const int head = local + 2 * static_cast<int>(blockIdx.x & 3);
  const bool is_v = (blockIdx.x & 4) != 0;
  int start, count;
  if (!new_tokens(a, b, &start, &count)) return;
  const PagedCache& pc = a.cache;
  const int P = 1 << pc.page_log2;
  const int pi = (start >> pc.page_log2) + static_cast<int>(blockIdx.x >> 3);  // of the sequence
  const int base = pi << pc.page_log2;  // the page's first index
  if (base >= start + count) return;
  const int s0 = start > base ? start - base : 0;  // slots [s0, s1) are new
  const int s1 = start + count - base < P ? start + count - base : P;
  const int t0 = base - start;  // token of slot 0
  const int page = __ldg(a.table + static_cast<int64_t>(b) * a.max_pages + pi);
  const uint16_t* src = (is_v ? a.v + b * a.v_batch : a.k + b * a.k_batch) + head * kHeadDim;
  const int64_t src_token = is_v ? a.v_token : a.k_token;

  uint4 keep[kTokens][2];  // this lane's chunks c and c+4
  const int mine = s0 + 4 * warp + sub;  // its first slot; the others 4 * warps apart
  auto load = [&](int s, uint4 (&w)[2]) {
    const uint4* p4 = reinterpret_cast<const uint4*>(src + (t0 + s) * src_token);
    w[0] = __ldg(p4 + c);
    w[1] = __ldg(p4 + c + 4);
  };
  auto value = [&](int s, const uint4 (&w)[2], bool exactly) {
    Halves x;
    x.unpack(w[0], w[1]);
    if (!is_v) {
      Turn turn;
      turn.load(table_row(a, b, t0 + s), c);
      if (exactly) {
        x.turn_exactly(turn);
      } else {
        x.turn(turn);
      }
    }
    return x;
  };
  // The same in 64 bits, this lane's pairs one after the other: products of a bf16 and a table
  // entry are exact there and overflow nothing, so only an infinite element gives an infinity.
  // (As rare as it is slow; it reads the token again, to leave the others their registers.)
  auto each_pair = [&](int s, auto&& use) {
    const uint16_t* x = src + (t0 + s) * src_token + 8 * c;
    const float2* row = is_v ? nullptr : table_row(a, b, t0 + s) + 8 * c;
#pragma unroll 1
    for (int e = 0; e < 8; ++e) {
      const double lo = bf16lo_to_f32(__ldg(x + e)), hi = bf16lo_to_f32(__ldg(x + e + 32));
      if (is_v) {
        use(e, lo, hi);
      } else {
        const float2 f = __ldg(row + e);
        use(e, lo * f.x - hi * f.y, hi * f.x + lo * f.y);
      }
    }
  };
#pragma unroll
  for (int i = 0; i < kTokens; ++i)
    if (mine + 4 * i * warps < s1) load(mine + 4 * i * warps, keep[i]);
  float top = 0.f;
#pragma unroll
  for (int i = 0; i < kTokens; ++i) {
    const int s = mine + 4 * i * warps;
    if (s >= s1) break;
    // (with the cheaper rotation, which is off by two or three ulps of the page's largest value)
    top = largest(value(s, keep[i], false), top);
  }
  const bool wide = !(top < kWide);
  // the largest finite value of this lane's tokens itself, in fp32
  auto exact_top = [&] {
    float t = 0.f;
#pragma unroll 1
    for (int s = mine; s < s1; s += 4 * warps)
      each_pair(s, [&](int, double lo, double hi) {
        // a value past fp32's range counts as fp32's largest: both take the largest scale
        if (fabs(lo) < HUGE_VAL) t = fmaxf(t, fminf(static_cast<float>(fabs(lo)), FLT_MAX));
        if (fabs(hi) < HUGE_VAL) t = fmaxf(t, fminf(static_cast<float>(fabs(hi)), FLT_MAX));
      });
    return t;
  };
  if (!paged_page_ok(page, pc.num_pages)) {
    if (threadIdx.x == 0) atomicOr(a.err, kErrPage);
    return;
  }
  // the largest of a head over the CTA, in every lane of the head
  auto of_page = [&](float t) {
    t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, 1));
    t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, 2));
    t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, 16));
    t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, 8));
    if (warps > 1) {
      if (c == 0 && sub == 0) tops[warp][local] = t;
      __syncthreads();  // and, the first time, every warp has read the scale
      for (int w = 0; w < warps; ++w) t = fmaxf(t, tops[w][local]);
    }
    return t;
  };
  // the scale that the page has, if it holds earlier tokens
  float* scale = (is_v ? pc.v_scale : pc.k_scale) + static_cast<int64_t>(page) * kNumKvHeads + head;
  const float before = s0 > 0 ? *scale : 0.f;
  top = of_page(top);
  // At a border the two rotations may lie on two sides. (Every warp has both heads' lanes, so
  // the whole CTA comes here or none does.)
  const bool again = !(top < kWide) || (!is_v && paged_near_border(__float_as_uint(top)));
  if (__any_sync(0xffffffffu, again)) {
    if (warps > 1) __syncthreads();
    top = of_page(exact_top());
  }
  __syncwarp();
  const float least = __uint_as_float(paged_scale_bits(__float_as_uint(top)));
  const float size = before >= least ? before : least;
  if (warp == 0 && c == 0 && sub == 0) *scale = size;
  uint8_t* dst = (is_v ? pc.v : pc.k) + page * pc.page_stride + head * pc.head_stride;
  if (size != before) {
    // it grew (for this lane's head): move the earlier tokens' codes
    const float f = before / size;
    for (int s = 4 * warp + sub; s < s0; s += 4 * warps) {
      uint4* row4 = reinterpret_cast<uint4*>(dst + s * pc.token_stride) + c;
      const uint4 w = *row4;
      *row4 = make_uint4(move_e4m3x4(w.x, f), move_e4m3x4(w.y, f), move_e4m3x4(w.z, f),
                         move_e4m3x4(w.w, f));
    }
  }
  const float inv = 1.f / size;
  if (wide) {
#pragma unroll 1
    for (int s = mine; s < s1; s += 4 * warps)
      each_pair(s, [&](int e, double lo, double hi) {
        uint8_t* at = dst + s * pc.token_stride + 8 * c + e;
        const uint32_t codes =
            pack_e4m3x2(static_cast<float>(lo * inv), static_cast<float>(hi * inv));
        at[0] = static_cast<uint8_t>(codes);
        at[32] = static_cast<uint8_t>(codes >> 8);
      });
    return;
  }
#pragma unroll
  for (int i = 0; i < kTokens; ++i) {
    const int s = mine + 4 * i * warps;
    if (s >= s1) break;
    const Halves x = value(s, keep[i], true);
    uint2* row2 = reinterpret_cast<uint2*>(dst + s * pc.token_stride);
    row2[c] = pack_e4m3x8(x.lo, inv);
    row2[c + 4] = pack_e4m3x8(x.hi, inv);
  }
}

}  // namespace

cudaError_t launch_paged_append(const PagedAppendArgs& a, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cfg.stream = stream;
  if (a.cache.fp8) {
    // pages that n tokens can touch, wherever in a page they start
    const int P = 1 << a.cache.page_log2;
    const int most = a.n < P ? a.n : P;  // new tokens in one page
    const unsigned pages = static_cast<unsigned>((a.n + P - 2) / P + 1);
    // Two tokens to a lane while all warps fit the GPU at once (32 to an SM), four beyond (2 x
    // 2048 in pages of 64 6.4 us, and 9.1 with four; 4 x 16384 51 us, and 59 with two. In
    // between two would still be better by a wave or so: 1 x 8192 9.3 us, 10.5 as it is).
    int warps = 1;
    while (warps < kAppendWarps && 8 * warps < most) warps *= 2;
    if (warps > 1 && static_cast<int64_t>(pages) * a.batch * 8 * warps > a.num_sms * 32) {
      warps = 1;
      while (warps < kAppendWarps && 16 * warps < most) warps *= 2;
    }
    cfg.gridDim = dim3(8 * pages, static_cast<unsigned>(a.batch));
    cfg.blockDim = dim3(static_cast<unsigned>(32 * warps));
    if (most <= 4 * warps) return cudaLaunchKernelEx(&cfg, append_e4m3_kernel<1>, a);
    if (most <= 8 * warps) return cudaLaunchKernelEx(&cfg, append_e4m3_kernel<2>, a);
    return cudaLaunchKernelEx(&cfg, append_e4m3_kernel<4>, a);
  }
  int warps = 1;
  while (warps < 8 && warps < a.n) warps *= 2;
  cfg.gridDim = dim3(static_cast<unsigned>((a.n + warps - 1) / warps),
                     static_cast<unsigned>(a.batch));
  cfg.blockDim = dim3(static_cast<unsigned>(32 * warps));
  return cudaLaunchKernelEx(&cfg, append_bf16_kernel, a);
}

}  // namespace gqa
