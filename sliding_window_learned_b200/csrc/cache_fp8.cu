// cache_fp8.cu -- an 8-bit paged key-value cache is written and read back:
//   append  bf16 K and V rows of packed sequences -> e4m3 codes and a scale
//           byte per (position, kv head), at the places the block table names
//   read    the same rows of the pools -> packed bf16
//
// Both are copies with a conversion, bound by HBM: a row moves 2D bytes on the
// bf16 side and D + 1 on the 8-bit side.  One pass: D/16 lanes hold one row's
// 16 channels each (two 16-byte halves, D/2 channels apart, so that every access
// of the row is contiguous), find the row's maximum by shuffles and store the
// codes, so nothing is read twice.
//
// The (row, head) vectors, heads fastest (the order both sides are contiguous
// in), go to the warps of one wave of blocks in turn, so that the warps that run
// together sweep through memory side by side.  A warp needs no other one: its
// lanes find the places of the next iteration's rows (the sequence by bisection
// of cu_seqlens, then the page) while this one's rows move, and hand them out by
// shuffles.  cu_seqlens and seqlens are staged in shared memory when they fit, so
// that a place is one global load, left in flight until it is used.
#include "e4m3.cuh"
#include "kernels.h"
#include "ptx.cuh"

namespace attnsink {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
// Blocks of the one wave, per SM.  Measured at 8 x 16 K rows, 8 kv heads, D = 128
// (4 / 3 / 2): append 122 / 127 / 152 us, read 146 / 143 / 126 us: the read's
// writes, two thirds of its bytes, do better from fewer places at a time.  (Short
// replays; back to back, under the power cap, append 139 and read 129 us.)  A read
// of few iterations is bound by latency instead and takes four (47 K rows of 2
// heads, D = 64: 9.5 us, 10.9 with two).
constexpr int kAppendBlocks = 4, kReadBlocks = 2, kShortReadBlocks = 4;
constexpr int kShortRead = 4;          // iterations
constexpr int kStageB = 1024;          // most sequences whose offsets and lengths are kept in shared memory

// kUnroll: vectors of K and of V that a lane has in flight.  Two, except where one
// gives every warp of the wave its first: then half as many for twice the warps
// (append of 64 rows of 4 heads 3.2 us against 3.8; of 131 K rows 163 against 122).
template <int D, int kUnroll>
struct Cfg {
  static constexpr int kLanes = D / 16;                    // lanes of one vector
  static constexpr int kPass = 32 / kLanes;                // vectors of a warp's pass
  static constexpr int kStep = kPass * kUnroll;            // and of its iteration
  static_assert(kStep <= 32, "one lane for each row of an iteration");
};

struct Place {
  int page;                            // pool page as the table has it; outside the pool: no place in the cache
  int at;                              // position within the page; -1: a row of no sequence
};

// Where packed row r belongs: the last rows of each sequence, in order.
__device__ __forceinline__ Place find_place(const CacheArgs &a, const int *cu, const int *seqlens, int64_t r) {
  Place pl{-1, -1};
  if (r >= a.T) return pl;
  int lo = 0, hi = a.B;                // last b in [0, B) with cu[b] <= r
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (cu[mid] <= r) lo = mid; else hi = mid;
  }
  const int64_t end = cu[lo + 1];
  if (cu[lo] > r || r >= end) return pl;
  const int64_t cap = static_cast<int64_t>(a.max_pages) << a.page_shift;
  const int64_t n = min(max(static_cast<int64_t>(seqlens[lo]), static_cast<int64_t>(0)), cap);
  const int64_t pos = n - (end - r);
  pl.at = 0;
  if (pos < 0) return pl;
  pl.page = a.block_table[lo * a.bt_s0 + (pos >> a.page_shift)];
  pl.at = static_cast<int>(pos & ((1 << a.page_shift) - 1));
  return pl;
}

// A warp's walk over the vectors: iteration by iteration, kStep of them.
struct Walk {
  const int *cu, *seqlens;
  int64_t row;                         // first row of the iteration
  int head;                            // and its first vector's head
  int left;                            // vectors from here to the end, at most kStep
  int64_t v;                           // first vector
  Place next;                          // lane l: place of row + l, not yet checked against the pool
};

// Stages the offsets and lengths (a block-wide barrier inside) and finds this
// warp's first iteration.
template <int kStep>
__device__ __forceinline__ Walk begin(const CacheArgs &a, int *stage) {
  Walk w;
  w.cu = a.cu_seqlens;
  w.seqlens = a.seqlens;
  if (a.B <= kStageB) {
    for (int i = threadIdx.x; i <= a.B; i += kThreads) {
      stage[i] = a.cu_seqlens[i];
      if (i < a.B) stage[kStageB + 1 + i] = a.seqlens[i];
    }
    w.cu = stage;
    w.seqlens = stage + kStageB + 1;
  }
  w.v = (static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5)) * kStep;
  w.row = w.v / a.Hkv;
  w.head = static_cast<int>(w.v - w.row * a.Hkv);
  w.left = static_cast<int>(min(a.T * a.Hkv - w.v, static_cast<int64_t>(kStep)));
  return w;
}

__device__ __forceinline__ void find_next(const CacheArgs &a, Walk *w) {
  w->next = find_place(a, w->cu, w->seqlens, w->row + (threadIdx.x & 31));
}

// Moves on by one iteration of every warp.
template <int kStep>
__device__ __forceinline__ void advance(const CacheArgs &a, Walk *w) {
  w->v += a.stride;
  w->row += a.stride_rows;
  w->head += a.stride_heads;
  if (w->head >= a.Hkv) {
    w->head -= a.Hkv;
    ++w->row;
  }
  w->left = static_cast<int>(min(a.T * a.Hkv - w->v, static_cast<int64_t>(kStep)));
}

// Row (from the iteration's first) and head of vector i of the iteration.
struct Vec {
  int row, head;
};
__device__ __forceinline__ Vec vec_of(const CacheArgs &a, const Walk &w, int i) {
  // (head + i) / Hkv by a multiplication: head + i < Hkv + 32 and Hkv <= 16384, so
  // the product's error stays below one part in Hkv
  Vec x;
  x.row = a.Hkv == 1 ? i : static_cast<int>(__umulhi(static_cast<unsigned>(w.head + i), a.hkv_inv));
  x.head = w.head + i - x.row * a.Hkv;
  return x;
}

// The place of the iteration's row `row`, from the lane that looked it up; page < 0
// where there is none.
__device__ __forceinline__ Place place_of(const CacheArgs &a, const Place &p, int row) {
  Place x;
  x.page = __shfl_sync(0xffffffffu, p.page, row);
  x.at = __shfl_sync(0xffffffffu, p.at, row);
  if (x.page >= a.npages) x.page = -1;
  return x;
}

// Packed maximum of two bf16 pairs' magnitudes (a NaN in either half stays one).
__device__ __forceinline__ uint32_t max_abs2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("{.reg .b32 x, y; abs.bf16x2 x, %1; abs.bf16x2 y, %2; max.NaN.bf16x2 %0, x, y;}" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint32_t max_abs8(const uint4 &x) { return max_abs2(max_abs2(x.x, x.y), max_abs2(x.z, x.w)); }

// The magnitudes of a pair with those of its non-finite halves zeroed.
__device__ __forceinline__ uint32_t finite_only(uint32_t x) {
  const uint32_t lo = x & 0x7FFFu, hi = x & 0x7FFF0000u;
  return (lo >= 0x7F80u ? 0u : lo) | (hi >= 0x7F800000u ? 0u : hi);
}

// A pair with its non-finite halves set to NaN.
__device__ __forceinline__ uint32_t inf_to_nan(uint32_t x) {
  const uint32_t lo = (x & 0x7FFFu) >= 0x7F80u ? 0x7FFFu : 0u;
  const uint32_t hi = (x & 0x7FFF0000u) >= 0x7F800000u ? 0x7FFF0000u : 0u;
  return x | lo | hi;
}

// A bf16 pair times `s` as two e4m3 codes.
__device__ __forceinline__ uint32_t codes_of(uint32_t x, float s) {
  return f32x2_to_e4m3x2(__uint_as_float(x << 16) * s, __uint_as_float(x & 0xFFFF0000u) * s);
}

struct Half2 {
  uint4 lo, hi;                        // 8 channels each, D/2 apart
};

__device__ __forceinline__ uint2 codes8(const uint4 &x, float s) {
  return make_uint2(codes_of(x.x, s) | codes_of(x.y, s) << 16, codes_of(x.z, s) | codes_of(x.w, s) << 16);
}
__device__ __forceinline__ uint4 finite8(const uint4 &x) {
  return make_uint4(finite_only(x.x), finite_only(x.y), finite_only(x.z), finite_only(x.w));
}
__device__ __forceinline__ uint4 nan8(const uint4 &x) {
  return make_uint4(inf_to_nan(x.x), inf_to_nan(x.y), inf_to_nan(x.z), inf_to_nan(x.w));
}

// Quantises one vector held by kLanes lanes: the codes of this lane's channels
// and the row's scale byte.  Every lane of the warp takes part.
template <int kLanes>
__device__ __forceinline__ void quantise(Half2 x, uint2 *lo, uint2 *hi, int *byte) {
  // (bf16 bits without the sign; NaN 0x7FFF)
  auto row_max = [](uint32_t m) {
#pragma unroll
    for (int o = 1; o < kLanes; o <<= 1) m = max_abs2(m, __shfl_xor_sync(0xffffffffu, m, o));
    return max(m & 0xFFFFu, m >> 16);
  };
  uint32_t m = row_max(max_abs2(max_abs8(x.lo), max_abs8(x.hi)));
  // NaN or infinity in some row of the warp (rare): the maxima again, over the
  // finite magnitudes alone, and infinities become NaN (the conversion would
  // saturate them to a finite code)
  if (__any_sync(0xffffffffu, m >= 0x7F80u)) {
    m = row_max(max_abs2(max_abs8(finite8(x.lo)), max_abs8(finite8(x.hi))));
    x.lo = nan8(x.lo);
    x.hi = nan8(x.hi);
  }
  *byte = row_scale_byte(m);
  const float s = row_inv_scale(*byte);
  *lo = codes8(x.lo, s);
  *hi = codes8(x.hi, s);
}

__device__ __forceinline__ uint4 load16(const __nv_bfloat16 *p) { return *reinterpret_cast<const uint4 *>(p); }
__device__ __forceinline__ uint2 load8(const uint8_t *p) { return *reinterpret_cast<const uint2 *>(p); }

template <int D, int kUnroll>
__global__ void __launch_bounds__(kThreads, kAppendBlocks) cache_append_kernel(const CacheArgs a) {
  using C = Cfg<D, kUnroll>;
  __shared__ int stage[2 * kStageB + 1];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;");
  Walk w = begin<C::kStep>(a, stage);
  __syncthreads();
  const int lane = threadIdx.x & 31, part = lane % C::kLanes, sub = lane / C::kLanes;
  if (w.left > 0) find_next(a, &w);
  while (w.left > 0) {
    Half2 k[kUnroll], x[kUnroll];
    Vec at[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int i = u * C::kPass + sub;
      at[u] = vec_of(a, w, i);
      k[u].lo = k[u].hi = x[u].lo = x[u].hi = make_uint4(0, 0, 0, 0);
      if (i >= w.left) continue;
      const __nv_bfloat16 *pk = a.k + (w.row + at[u].row) * a.k_s[0] + at[u].head * a.k_s[1] + part * 8;
      const __nv_bfloat16 *pv = a.v + (w.row + at[u].row) * a.v_s[0] + at[u].head * a.v_s[1] + part * 8;
      k[u].lo = load16(pk);
      k[u].hi = load16(pk + D / 2);
      x[u].lo = load16(pv);
      x[u].hi = load16(pv + D / 2);
    }
    const Place place = w.next;
    const int left = w.left;
    advance<C::kStep>(a, &w);
    if (w.left > 0) find_next(a, &w);
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      if (u * C::kPass >= left) break;                           // (warp-uniform)
      const int i = u * C::kPass + sub;
      // (lanes behind the last vector take part in the shuffles)
      const Place pl = place_of(a, place, i < left ? at[u].row : 0);
      uint2 k0, k1, v0, v1;
      int kb, vb;
      quantise<C::kLanes>(k[u], &k0, &k1, &kb);
      quantise<C::kLanes>(x[u], &v0, &v1, &vb);
      if (i >= left || pl.page < 0) continue;
      const int64_t pg = pl.page;
      uint8_t *pk = a.kpages + pg * a.kp_s[0] + pl.at * a.kp_s[1] + at[u].head * a.kp_s[2] + part * 8;
      uint8_t *pv = a.vpages + pg * a.vp_s[0] + pl.at * a.vp_s[1] + at[u].head * a.vp_s[2] + part * 8;
      *reinterpret_cast<uint2 *>(pk) = k0;
      *reinterpret_cast<uint2 *>(pk + D / 2) = k1;
      *reinterpret_cast<uint2 *>(pv) = v0;
      *reinterpret_cast<uint2 *>(pv + D / 2) = v1;
      if (part == 0) a.kscales[pg * a.ks_s[0] + at[u].head * a.ks_s[1] + pl.at] = static_cast<uint8_t>(kb);
      if (part == 1) a.vscales[pg * a.vs_s[0] + at[u].head * a.vs_s[1] + pl.at] = static_cast<uint8_t>(vb);
    }
  }
}

// Eight codes times a scale as packed bf16.  f32 holds the product exactly (or
// rounds a scale no append writes), and so does bf16 for every written scale.
__device__ __forceinline__ uint4 values_of(const uint2 &c, float s) {
  const uint2 a = e4m3x4_to_f16x2x2(c.x), b = e4m3x4_to_f16x2x2(c.y);
  const uint32_t h[4] = {a.x, a.y, b.x, b.y};
  uint32_t r[4];
#pragma unroll
  for (int t = 0; t < 4; ++t) {
    float lo, hi;
    asm("{.reg .b16 l, h; mov.b32 {l, h}, %2; cvt.f32.f16 %0, l; cvt.f32.f16 %1, h;}"
        : "=f"(lo), "=f"(hi)
        : "r"(h[t]));
    r[t] = pack_bf16x2(lo * s, hi * s);
  }
  return make_uint4(r[0], r[1], r[2], r[3]);
}

template <int D, int kUnroll>
__global__ void __launch_bounds__(kThreads) cache_read_kernel(const CacheArgs a) {
  using C = Cfg<D, kUnroll>;
  __shared__ int stage[2 * kStageB + 1];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;");
  Walk w = begin<C::kStep>(a, stage);
  __syncthreads();
  const int lane = threadIdx.x & 31, part = lane % C::kLanes, sub = lane / C::kLanes;
  if (w.left > 0) find_next(a, &w);
  while (w.left > 0) {
    const Place place = w.next;
    uint2 k0[kUnroll], k1[kUnroll], v0[kUnroll], v1[kUnroll];
    uint32_t kb[kUnroll], vb[kUnroll];
    int64_t row[kUnroll];              // -1: nothing is written
    int head[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int i = u * C::kPass + sub;
      const Vec at = vec_of(a, w, i);
      const Place pl = place_of(a, place, i < w.left ? at.row : 0);
      // rows of no sequence stay as they are; a row without a place reads as zeros
      row[u] = i < w.left && pl.at >= 0 ? w.row + at.row : -1;
      head[u] = at.head;
      k0[u] = k1[u] = v0[u] = v1[u] = make_uint2(0, 0);
      kb[u] = vb[u] = 127;
      if (i >= w.left || pl.page < 0) continue;
      const int64_t pg = pl.page;
      const uint8_t *pk = a.kpages + pg * a.kp_s[0] + pl.at * a.kp_s[1] + at.head * a.kp_s[2] + part * 8;
      const uint8_t *pv = a.vpages + pg * a.vp_s[0] + pl.at * a.vp_s[1] + at.head * a.vp_s[2] + part * 8;
      k0[u] = load8(pk);
      k1[u] = load8(pk + D / 2);
      v0[u] = load8(pv);
      v1[u] = load8(pv + D / 2);
      kb[u] = a.kscales[pg * a.ks_s[0] + at.head * a.ks_s[1] + pl.at];
      vb[u] = a.vscales[pg * a.vs_s[0] + at.head * a.vs_s[1] + pl.at];
    }
    advance<C::kStep>(a, &w);
    if (w.left > 0) find_next(a, &w);
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      if (row[u] < 0) continue;
      const float ks = scale_value(kb[u]), vs = scale_value(vb[u]);
      __nv_bfloat16 *pk = a.k_out + row[u] * a.k_s[0] + head[u] * a.k_s[1] + part * 8;
      __nv_bfloat16 *pv = a.v_out + row[u] * a.v_s[0] + head[u] * a.v_s[1] + part * 8;
      *reinterpret_cast<uint4 *>(pk) = values_of(k0[u], ks);
      *reinterpret_cast<uint4 *>(pk + D / 2) = values_of(k1[u], ks);
      *reinterpret_cast<uint4 *>(pv) = values_of(v0[u], vs);
      *reinterpret_cast<uint4 *>(pv + D / 2) = values_of(v1[u], vs);
    }
  }
}

template <int D, int kUnroll>
cudaError_t launch_unrolled(CacheArgs a, bool append, int blocks_per_sm, int sms, cudaStream_t stream) {
  using C = Cfg<D, kUnroll>;
  auto kern = append ? cache_append_kernel<D, kUnroll> : cache_read_kernel<D, kUnroll>;
  // one wave of blocks, or as many as have a vector
  const int64_t steps = (a.T * a.Hkv + C::kStep - 1) / C::kStep;
  const int64_t need = (steps + kWarps - 1) / kWarps, wave = static_cast<int64_t>(sms) * blocks_per_sm;
  const int64_t blocks = need < wave ? need : wave;
  a.stride = blocks * kWarps * C::kStep;
  a.stride_rows = a.stride / a.Hkv;
  a.stride_heads = static_cast<int>(a.stride - a.stride_rows * a.Hkv);
  a.hkv_inv = a.Hkv == 1 ? 0 : static_cast<uint32_t>(0x100000000ull / static_cast<uint64_t>(a.Hkv) + 1);
  // (launched with programmatic dependence, as the decode that may follow: its
  // blocks come up while the kernel before it ends)
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(blocks));
  cfg.blockDim = dim3(kThreads);
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, a);
}

template <int D>
cudaError_t launch(const CacheArgs &a, bool append, int sms, cudaStream_t stream) {
  const int64_t total = a.T * a.Hkv, warps = static_cast<int64_t>(sms) * kWarps;
  const bool short_read = total <= warps * kShortReadBlocks * kShortRead * Cfg<D, 2>::kStep;
  const int blocks = append ? kAppendBlocks : short_read ? kShortReadBlocks : kReadBlocks;
  if (total <= warps * blocks * Cfg<D, 1>::kStep) return launch_unrolled<D, 1>(a, append, blocks, sms, stream);
  return launch_unrolled<D, 2>(a, append, blocks, sms, stream);
}

}  // namespace

cudaError_t launch_cache(const CacheArgs &a, bool append, int sms, cudaStream_t stream) {
  switch (a.D) {
    case 64: return launch<64>(a, append, sms, stream);
    case 128: return launch<128>(a, append, sms, stream);
    case 256: return launch<256>(a, append, sms, stream);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace attnsink
