// cache_fp8.cu -- an 8-bit paged key-value cache is written and read back:
//   append  bf16 K and V rows of packed sequences -> e4m3 codes and a scale
//           byte per (position, kv head), at the places the block table names
//   read    the same rows of the pools -> packed bf16
//
// Both are copies with a conversion, bound by HBM: a row moves 2D bytes on the
// bf16 side and D + 1 on the 8-bit side.  One pass: D/8 lanes hold one row's
// 8 channels each in registers, find the row's maximum by shuffles and store
// the codes, so nothing is read twice.  Every thread has kUnroll rows of K and
// of V in flight.
//
// A block takes a run of consecutive (row, head) vectors, heads fastest (the
// order both sides are contiguous in).  Its rows' places are found once, in
// shared memory: the sequence of a row by bisection of cu_seqlens (staged in
// shared memory when it fits, so that the probes are not dependent global
// loads), then its page.  The append issues its row loads before that, so the
// two latencies overlap.
#include "e4m3.cuh"
#include "kernels.h"
#include "ptx.cuh"

namespace attnsink {
namespace {

constexpr int kThreads = 256;
constexpr int kUnroll = 4;             // vectors of K and of V per thread
constexpr int kCuStage = 1024;         // longest cu_seqlens kept in shared memory

template <int D>
struct Cfg {
  static constexpr int kLanes = D / 8;                     // lanes of one vector
  static constexpr int kPass = kThreads / kLanes;          // vectors per pass of the block
  static constexpr int kVecs = kPass * kUnroll;            // vectors per block
  static_assert(kVecs <= kThreads, "one thread finds each row's place");
};

struct Place {
  int page;                            // pool page, -1: the row has no place
  int at;                              // position within the page
};

// Where packed row r belongs: the last rows of each sequence, in order.
__device__ __forceinline__ Place find_place(const CacheArgs &a, const int *cu, int64_t r) {
  Place pl{-1, 0};
  int lo = 0, hi = a.B;                // last b in [0, B) with cu[b] <= r
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (cu[mid] <= r) lo = mid; else hi = mid;
  }
  const int64_t end = cu[lo + 1];
  if (cu[lo] > r || r >= end) return pl;
  const int64_t cap = static_cast<int64_t>(a.max_pages) << a.page_shift;
  const int64_t n = min(max(static_cast<int64_t>(a.seqlens[lo]), static_cast<int64_t>(0)), cap);
  const int64_t pos = n - (end - r);
  if (pos < 0) return pl;
  const int page = a.block_table[lo * a.bt_s0 + (pos >> a.page_shift)];
  if (page < 0 || page >= a.npages) return pl;
  pl.page = page;
  pl.at = static_cast<int>(pos & ((1 << a.page_shift) - 1));
  return pl;
}

// Fills places[] for the rows [r0, r0 + nr) of this block; ends with a barrier.
__device__ __forceinline__ void find_places(const CacheArgs &a, int64_t r0, int nr, int *cu_s, Place *places) {
  const int *cu = a.cu_seqlens;
  if (a.B < kCuStage) {
    for (int i = threadIdx.x; i <= a.B; i += kThreads) cu_s[i] = a.cu_seqlens[i];
    cu = cu_s;
  }
  __syncthreads();
  if (static_cast<int>(threadIdx.x) < nr) places[threadIdx.x] = find_place(a, cu, r0 + threadIdx.x);
  __syncthreads();
}

// Largest magnitude (bf16 bits without the sign) of 8 packed bf16.
__device__ __forceinline__ uint32_t max_bits(const uint4 &x) {
  const uint32_t m = 0x7FFF7FFFu;
  const uint32_t t = __vmaxu2(__vmaxu2(x.x & m, x.y & m), __vmaxu2(x.z & m, x.w & m));
  return max(t & 0xFFFFu, t >> 16);
}

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

// Quantises one vector held by kLanes lanes (8 channels each): the codes of
// this lane's channels and the row's scale byte.
template <int kLanes>
__device__ __forceinline__ uint2 quantise(uint4 x, int *byte) {
  uint32_t m = max_bits(x);
#pragma unroll
  for (int o = 1; o < kLanes; o <<= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
  // NaN or infinity in some row of the warp (rare): the maxima again, over the
  // finite magnitudes alone, and infinities become NaN (the conversion would
  // saturate them to a finite code)
  if (__any_sync(0xffffffffu, m >= 0x7F80u)) {
    m = max_bits(make_uint4(finite_only(x.x), finite_only(x.y), finite_only(x.z), finite_only(x.w)));
#pragma unroll
    for (int o = 1; o < kLanes; o <<= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
    x = make_uint4(inf_to_nan(x.x), inf_to_nan(x.y), inf_to_nan(x.z), inf_to_nan(x.w));
  }
  *byte = row_scale_byte(m);
  const float s = row_inv_scale(*byte);
  return make_uint2(codes_of(x.x, s) | codes_of(x.y, s) << 16, codes_of(x.z, s) | codes_of(x.w, s) << 16);
}

template <int D>
__global__ void __launch_bounds__(kThreads) cache_append_kernel(const CacheArgs a) {
  using C = Cfg<D>;
  __shared__ int cu_s[kCuStage];
  __shared__ Place places[kThreads];
  const int64_t v0 = static_cast<int64_t>(blockIdx.x) * C::kVecs;
  const int64_t total = a.T * a.Hkv;
  const int nv = static_cast<int>(min(total - v0, static_cast<int64_t>(C::kVecs)));
  const int64_t r0 = v0 / a.Hkv;
  const int h0 = static_cast<int>(v0 - r0 * a.Hkv);
  const int nr = (h0 + nv - 1) / a.Hkv + 1;
  const int lane = threadIdx.x % C::kLanes;
  uint4 k[kUnroll], v[kUnroll];
  int row[kUnroll], head[kUnroll];
#pragma unroll
  for (int u = 0; u < kUnroll; ++u) {
    const int i = u * C::kPass + static_cast<int>(threadIdx.x) / C::kLanes;
    row[u] = (h0 + i) / a.Hkv;
    head[u] = h0 + i - row[u] * a.Hkv;
    k[u] = v[u] = make_uint4(0, 0, 0, 0);
    if (i < nv) {
      const int64_t r = r0 + row[u];
      k[u] = __ldcs(reinterpret_cast<const uint4 *>(a.k + r * a.k_s[0] + head[u] * a.k_s[1] + lane * 8));
      v[u] = __ldcs(reinterpret_cast<const uint4 *>(a.v + r * a.v_s[0] + head[u] * a.v_s[1] + lane * 8));
    } else {
      row[u] = -1;
    }
  }
  find_places(a, r0, nr, cu_s, places);
#pragma unroll
  for (int u = 0; u < kUnroll; ++u) {
    // (every lane takes part in the shuffles, whether its vector is kept or not)
    int kb, vb;
    const uint2 kc = quantise<C::kLanes>(k[u], &kb);
    const uint2 vc = quantise<C::kLanes>(v[u], &vb);
    if (row[u] < 0) continue;
    const Place pl = places[row[u]];
    if (pl.page < 0) continue;
    const int h = head[u];
    *reinterpret_cast<uint2 *>(a.kpages + pl.page * a.kp_s[0] + pl.at * a.kp_s[1] + h * a.kp_s[2] + lane * 8) = kc;
    *reinterpret_cast<uint2 *>(a.vpages + pl.page * a.vp_s[0] + pl.at * a.vp_s[1] + h * a.vp_s[2] + lane * 8) = vc;
    if (lane == 0) {
      a.kscales[pl.page * a.ks_s[0] + h * a.ks_s[1] + pl.at] = static_cast<uint8_t>(kb);
      a.vscales[pl.page * a.vs_s[0] + h * a.vs_s[1] + pl.at] = static_cast<uint8_t>(vb);
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

template <int D>
__global__ void __launch_bounds__(kThreads) cache_read_kernel(const CacheArgs a) {
  using C = Cfg<D>;
  __shared__ int cu_s[kCuStage];
  __shared__ Place places[kThreads];
  const int64_t v0 = static_cast<int64_t>(blockIdx.x) * C::kVecs;
  const int64_t total = a.T * a.Hkv;
  const int nv = static_cast<int>(min(total - v0, static_cast<int64_t>(C::kVecs)));
  const int64_t r0 = v0 / a.Hkv;
  const int h0 = static_cast<int>(v0 - r0 * a.Hkv);
  const int nr = (h0 + nv - 1) / a.Hkv + 1;
  const int lane = threadIdx.x % C::kLanes;
  find_places(a, r0, nr, cu_s, places);
  // rows past the last sequence (or before the first) stay as they are
  const int64_t first = a.cu_seqlens[0], last = a.cu_seqlens[a.B];
  uint2 kc[kUnroll], vc[kUnroll];
  uint32_t kb[kUnroll], vb[kUnroll];
#pragma unroll
  for (int u = 0; u < kUnroll; ++u) {
    const int i = u * C::kPass + static_cast<int>(threadIdx.x) / C::kLanes;
    const int row = (h0 + i) / a.Hkv, h = h0 + i - row * a.Hkv;
    kc[u] = vc[u] = make_uint2(0, 0);
    kb[u] = vb[u] = 127;
    if (i >= nv) continue;
    const Place pl = places[row];
    if (pl.page < 0) continue;
    kc[u] = __ldcs(reinterpret_cast<const uint2 *>(a.kpages + pl.page * a.kp_s[0] + pl.at * a.kp_s[1] +
                                                   h * a.kp_s[2] + lane * 8));
    vc[u] = __ldcs(reinterpret_cast<const uint2 *>(a.vpages + pl.page * a.vp_s[0] + pl.at * a.vp_s[1] +
                                                   h * a.vp_s[2] + lane * 8));
    kb[u] = a.kscales[pl.page * a.ks_s[0] + h * a.ks_s[1] + pl.at];
    vb[u] = a.vscales[pl.page * a.vs_s[0] + h * a.vs_s[1] + pl.at];
  }
#pragma unroll
  for (int u = 0; u < kUnroll; ++u) {
    const int i = u * C::kPass + static_cast<int>(threadIdx.x) / C::kLanes;
    const int row = (h0 + i) / a.Hkv, h = h0 + i - row * a.Hkv;
    const int64_t r = r0 + row;
    if (i >= nv || r < first || r >= last) continue;
    // (a row without a place reads as zeros)
    *reinterpret_cast<uint4 *>(a.k_out + r * a.k_s[0] + h * a.k_s[1] + lane * 8) = values_of(kc[u], scale_value(kb[u]));
    *reinterpret_cast<uint4 *>(a.v_out + r * a.v_s[0] + h * a.v_s[1] + lane * 8) = values_of(vc[u], scale_value(vb[u]));
  }
}

template <int D>
cudaError_t launch(const CacheArgs &a, bool append, cudaStream_t stream) {
  const int64_t total = a.T * a.Hkv;
  const int64_t blocks = (total + Cfg<D>::kVecs - 1) / Cfg<D>::kVecs;
  if (blocks > 0x7FFFFFFF) return cudaErrorInvalidValue;
  if (append)
    cache_append_kernel<D><<<static_cast<unsigned>(blocks), kThreads, 0, stream>>>(a);
  else
    cache_read_kernel<D><<<static_cast<unsigned>(blocks), kThreads, 0, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_cache(const CacheArgs &a, bool append, cudaStream_t stream) {
  switch (a.D) {
    case 64: return launch<64>(a, append, stream);
    case 128: return launch<128>(a, append, stream);
    case 256: return launch<256>(a, append, stream);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace attnsink
