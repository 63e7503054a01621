// decode_paged_fp8.cu -- single-token decode over the 8-bit paged cache
// (e4m3 codes, one power-of-two scale per position and kv head), with the
// causal window and the learned sink.
//
// With x_j = scale*log2e * 2^ek_j * <q, ck_j> (codes ck, scale exponents ek, ev):
//   O = sum_j 2^x_j 2^ev_j cv_j / ( sum_j 2^x_j + 2^(sink*log2e) )
// The value scales differ from key to key over up to 236 binades, so folding
// them into P would overflow or flush its f16.  The numerator therefore keeps
// a reference of its own, over y_j = x_j + ev_j, beside the softmax's over x_j:
//   N = sum_j 2^(y_j - m) cv_j,  L = sum_j 2^(x_j - M),  O = N 2^(m - M) / L.
// Both references move lazily (only when an exponent would exceed 2^8), which a
// warp vote decides: the common tile needs no shuffle.  m is held as m - M: with the
// two apart, a logit's rounding scaled the output (12 % at logits of 2^20).
//
// Two launches, no host synchronisation:
//   split    persistent, one CTA per SM.  Every CTA reads the lengths and finds
//            its own share: the key tiles of all sequences, one after another,
//            are cut into E equal spans ("teams"), and one item is (span, kv
//            head), heads fastest, so that the CTAs that run together read the
//            heads of the same positions (whole DRAM bursts).  A span may
//            end one sequence and begin others; a sequence that lies in one span
//            is finished there (sink included), one that is cut leaves a partial
//            (O_s, LSE_s) per span.  Launched with programmatic dependence too:
//            its CTAs set up while the kernel before them ends.
//   combine  merges the spans of each cut sequence, in order, and adds the sink
//            once; writes zeros for empty sequences.  Launched with programmatic
//            dependence: its blocks are resident before the split ends.
// At most two partials exist per span, whatever the lengths.  Where all sequences
// are short, items are whole sequences and the split is the only launch.
//
// Inside the split, twelve (D = 256: eight) consumer warps and four producer warps:
//   consumers  a warp owns 16 (D = 64: 32) keys of every tile.  e4m3 is converted
//              to f16 in registers (exact) and both products run on warp-level f16
//              MMAs: S^T = K q^T and O^T += V^T P^T, heads the N = 8 dimension, q
//              in f16 under a power-of-two scale per head.
//   producers  find the CTA's share; stream the tiles into a ring of stages (a lane
//              looks after 16 keys' page: boxes of min(page, 64) positions x all D
//              channels of a head by TMA, the 16 scale bytes by a 16-byte
//              asynchronous copy, all counted on the stage's barrier); one of
//              them prepares each piece's q; and all four merge the consumers'
//              states at the end of a piece while the consumers go on.
//
// Bound by HBM at long contexts: D + 1 bytes per key, kv head and K or V.  64
// sequences of 4 K..131 K keys, Hq32 Hkv4 D128, 256-position pages, calls back to
// back: 774 us, 6.0 TB/s (0.91 of the measured copy rate), with the clock at 1.5 GHz
// under the power cap; 640 us in short replays at 1.9 GHz, as all figures from here
// on.  8 of them 109 us (118 back to back), where the start (2 us to the first
// copies, then every CTA's first stages at once) and the end show.  With 16 heads a
// group the consumers' chain of dependent instructions bounds it: 5.6 TB/s.  Tried and dropped, each against the
// version it was tried on: K's codes straight into e4m3 MMAs with q as two e4m3
// terms (a quarter fewer instructions, but those MMAs' latency is longer: 643 ->
// 720 us, 16 heads 503 -> 667); the consumers as two groups that take tiles in turn
// with two key blocks a warp (110 -> 113 us, D = 64 204 -> 304); one producer warp
// (its lanes' TMA copies are issued one after another: pages of 16 positions 119 us
// against 74); the merge as a function of its own (its spills cost 2.4 us of launch
// time).
#include <math.h>

#include <type_traits>

#include "e4m3.cuh"
#include "kernels.h"
#include "ptx.cuh"

namespace attnsink {
namespace {

constexpr uint32_t kBarInit = 1;      // named barrier: every thread, once
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kLog2e = 1.4426950408889634f;
enum : int { kWhereFull = 401, kWhereEmpty = 402, kWhereMerge = 403, kWhereAlign = 404 };

// The numerator's P is f16, up to 2^15: kHeadroom keeps it as far from the
// subnormals as the lazy reference (exponents up to kLazy above it) allows.
constexpr float kLazy = 8.0f;
constexpr float kHeadroom = 7.0f;
constexpr float kNoMax = -0x1.fffffep127f;   // a reference nothing was seen against: the lowest f32

// S = K q^T reaches 2^31 (q in f16 up to 2^14), a key's scale 2^119: their product is
// taken under 2^-24, and the softmax scale, which undoes q's power of two, over it.
// Logits that fit f32 then pass through no intermediate that does not.  (Where a
// head's queries are so large, above 2^119, that its softmax scale would overflow,
// the piece goes without the factor: large keys overflow its logits themselves.)
constexpr float kDown = 0x1p-24f;

// ------------------------------------------------------------- workspace
struct Workspace {
  size_t off_info, off_lse, off_o, total;
};

__host__ __device__ inline size_t align256(size_t x) { return (x + 255) & ~static_cast<size_t>(255); }

// Spans at most: as many as give every SM an item, or the smallest number of
// rounds (up to four) that leaves at most a tenth of the SMs idle.
int max_teams(int Hkv, int sms) {
  int best = 1;
  double used = 0;
  for (int w = 1; w <= 4; ++w) {
    const int t = static_cast<int>(static_cast<int64_t>(w) * sms / Hkv);
    if (t < 1) continue;
    const double u = static_cast<double>(t) * Hkv / (static_cast<double>(w) * sms);
    if (u > used + 0.05) {
      used = u;
      best = t;
    }
    if (used >= 0.9) break;
  }
  return best;
}

Workspace layout(const PagedFp8Args &a, int teams) {
  Workspace w;
  size_t off = 0;
  w.off_info = off;                                     // [teams] int2 (first sequence cut here, last span), [teams] = E
  off = align256(off + sizeof(int2) * (teams + 1));
  w.off_lse = off;                                      // [2 * teams][Hq]
  off = align256(off + sizeof(float) * 2 * teams * a.Hq);
  w.off_o = off;                                        // [2 * teams][Hq][D]
  off = align256(off + sizeof(float) * 2 * teams * a.Hq * a.D);
  w.total = off;
  return w;
}

// Where no sequence can have more tiles than this (a short window or a short
// table), nothing is cut: an item is a sequence's kv head, there is no plan, no
// workspace and no combine launch.  4 kv heads, D = 128, whole against cut (both
// before the overlapped start, which takes 0.6 us off either): one sequence in a
// window of 513 (three tiles) 8.7 and 9.6 us, 64 of them 15.5 and 19.2; at seven tiles (a window of 1300) it turns with the batch: two sequences
// 12.3 and 11.1, sixteen 13.4 and 14.9.
constexpr int kWholeTiles = 4;
constexpr int tile_keys(int D) { return D == 64 ? 384 : D == 128 ? 192 : 128; }
bool takes_whole(const PagedFp8Args &a) {
  const int64_t cap = static_cast<int64_t>(a.max_pages) * a.page;
  const int64_t keys = (a.W < cap ? a.W : cap) + (a.page < 64 ? a.page : 64) - 1;   // (from a box's start)
  return keys <= kWholeTiles * tile_keys(a.D) && static_cast<int64_t>(a.B) * a.Hkv <= (1 << 30);
}

struct Params {
  PagedFp8Args a;
  int G, teams, page_shift, box_rows, box_shift;
  int out8;                              // rows of out keep 8-byte alignment
  int whole;                             // nothing is cut (kWholeTiles)
  float scale_log2;
  int2 *info;
  float *lse_part, *o_part;
};

// Keys [lo, n) of a sequence in tiles of TK starting at lo rounded down to a box.
struct Range {
  int n, vis0, start, tiles;
};
template <int TK>
__device__ __forceinline__ Range range_of(const Params &p, int seqlen) {
  Range r;
  const long long cap = static_cast<long long>(p.a.max_pages) << p.page_shift;
  r.n = static_cast<int>(min(static_cast<long long>(max(seqlen, 0)), cap));
  r.vis0 = max(0, r.n - p.a.W);
  r.start = r.vis0 & ~(p.box_rows - 1);
  r.tiles = (r.n - r.start + TK - 1) / TK;
  return r;
}

struct StageInfo {
  int b, hk, dest, nvalid;             // dest: partial slot, or -1: the sequence is finished here
  int nskip, flags, pad0, pad1;        // flags: 1 first tile of a piece, 2 last tile, 4 end of work
};

// A piece's partial states of one head tile, handed to the producer warps.
struct MergeUnit {
  int b, hk, dest, nt;                 // as StageInfo; head tile
  int stage, last, pad0, pad1;         // the stage that holds O; the piece's last unit
};

template <int D, int NT>
struct Cfg {
  // Consumer warps: twelve hide the conversion's latency; at D = 256 eight, as
  // many as three 64 KB stages allow.
  static constexpr int kCW = D == 256 ? 8 : 12;
  // Two head tiles at D = 128: the q fragments stay in shared memory, so that
  // twelve warps keep within 128 registers each.
  static constexpr bool kQInSmem = NT == 2 && D >= 128;
  // 16-key blocks of a warp per tile: two at D = 64, whose rows are half as long
  // (the same bytes per stage, and two independent chains of work in flight).
  static constexpr int kKB = D == 64 ? 2 : 1;
  static constexpr int kTK = 16 * kKB * kCW;
  // Producer warps: each issues the copies of its share of the tile's keys (a
  // warp issues its lanes' TMA copies one after another).
  static constexpr int kPW = 4;
  static constexpr int kShare = kTK / 16 / kPW;             // 16-key chunks of one producer warp
  static constexpr int kWarps = kCW + kPW;
  static constexpr int kThreads = kWarps * 32;
  static constexpr int kInner = D < 128 ? D : 128;          // bytes of a swizzled row
  static constexpr int kChunks = D / kInner;
  static constexpr int kTileBytes = kTK * D;
  static constexpr int kStageBytes = 2 * kTileBytes;        // K then V
  static constexpr int kScaleBytes = 2 * kTK;               // per stage: K then V
  // a piece's q as B fragments [k-step][head tile][lane], its heads' scales and kDown's factor.
  // One slot more than stages: when a piece's first tile has its stage, the piece
  // kQSlots before has been released to its last tile, so a slot needs no barrier
  // to say that it is free.
  static constexpr int kQScale = (D / 16) * NT * 32 * 8;
  static constexpr int kQSlot = kQScale + NT * 8 * 4 + 8;
  static constexpr int kQSlots = 5;
  static constexpr int kQBytes = (kQSlots * kQSlot + 127) / 128 * 128;
  static constexpr int kFixed = kQBytes + 3 * kCW * 8 * 4 + 1024;
  static constexpr int kStagesRaw = (232448 - kFixed) / (kStageBytes + kScaleBytes + 64);
  static constexpr int kStages = kStagesRaw > kQSlots - 1 ? kQSlots - 1 : kStagesRaw;
  static constexpr int kQOffset = kStages * kStageBytes;
  static constexpr int kScaleOffset = kQOffset + kQBytes;
  static constexpr int kInfoOffset = kScaleOffset + (kStages * kScaleBytes + 127) / 128 * 128;
  // stage infos and barriers; the consumers' meeting, merge and q barriers; the
  // merge unit, (m, M, L) per warp and head, abort flag
  static constexpr int kTail = kStages * (32 + 16) + (3 + kQSlots) * 8 + 32 + 3 * kCW * 8 * 4 + 32;
  static constexpr int kSmemBytes = kInfoOffset + kTail;
  static_assert(kTK == tile_keys(D), "tile size");
  static_assert(kStages >= 3, "ring");
  static_assert(kSmemBytes <= 232448, "shared-memory budget");
  static_assert(kCW * 8 * D * 4 <= kStageBytes, "one merge pass fits a stage");
  static_assert(kCW % kPW == 0, "the producer warps arrive for the consumers after a merge");
  static_assert(kShare * kPW * 16 == kTK && kShare <= 16, "one lane per 16 keys of K and of V");
};

__device__ __forceinline__ bool warp_wait(uint64_t *bar, uint32_t parity, const WaitCtx &ctx, int where) {
  const bool r = mbar_wait(bar, parity, ctx, where);
  return __all_sync(0xffffffffu, r);
}

// Whether the phase with the given parity is over, without waiting.
__device__ __forceinline__ bool mbar_test_wait(uint64_t *bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.test_wait.parity.acquire.cta.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(smem_u32(bar)), "r"(parity)
      : "memory");
  return ok != 0;
}

__device__ __forceinline__ void mbar_arrive_n(uint64_t *bar, uint32_t n) {
  asm volatile("mbarrier.arrive.release.cta.shared::cta.b64 _, [%0], %1;" ::"r"(smem_u32(bar)), "r"(n) : "memory");
}

// Quotient of non-negative values, by the 32-bit divider where they fit.
__device__ __forceinline__ long long div_ll(long long a, long long b) {
  if (((a | b) >> 32) == 0) return static_cast<uint32_t>(a) / static_cast<uint32_t>(b);
  return a / b;
}

// 16 bytes global -> shared, or 16 zero bytes when !valid (nothing is read).
__device__ __forceinline__ void copy16_async(void *dst, const void *src, bool valid) {
  const int n = valid ? 16 : 0;
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(dst)), "l"(src), "r"(n) : "memory");
}
// The barrier gets one arrival when this thread's copies so far have landed.
__device__ __forceinline__ void copy_async_arrive(uint64_t *bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}
__device__ __forceinline__ void copy_async_wait_all() { asm volatile("cp.async.wait_all;" ::: "memory"); }

__device__ __forceinline__ uint32_t f32x2_to_f16x2(uint32_t bf, float s) {
  return pack_f16x2(__uint_as_float(bf << 16) * s, __uint_as_float(bf & 0xFFFF0000u) * s);
}

template <int D, int NT>
__global__ void __launch_bounds__(Cfg<D, NT>::kThreads, 1)
    paged_fp8_split_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                           const __grid_constant__ Params p) {
  using C = Cfg<D, NT>;
  // (128-byte swizzled boxes need 1024-byte aligned addresses; aligning by hand
  // would hide from the compiler that this is shared memory)
  extern __shared__ __align__(1024) uint8_t smem[];
  if (reinterpret_cast<uintptr_t>(smem) & 1023u) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (threadIdx.x == 0) report_launch_error(p.a.status, kWhereAlign);
    return;
  }
  // (whole: the kernel behind may come up from here on, 8.35 -> 8.05 us a call; where
  // it is the combine, which reads before it waits, only behind this one's wait)
  if (p.whole) asm volatile("griddepcontrol.launch_dependents;");
  StageInfo *info = reinterpret_cast<StageInfo *>(smem + C::kInfoOffset);
  uint64_t *full = reinterpret_cast<uint64_t *>(info + C::kStages);
  uint64_t *empty = full + C::kStages;
  uint64_t *meet = empty + C::kStages;       // the consumers are done with a piece's last stage
  uint64_t *merge_full = meet + 1;           // a merge unit is in shared memory
  uint64_t *merge_free = merge_full + 1;     // and has been read
  uint64_t *q_full = merge_free + 1;         // [kQSlots] a piece's q is in its slot
  MergeUnit *unit = reinterpret_cast<MergeUnit *>(q_full + C::kQSlots);
  float *merge_d = reinterpret_cast<float *>(unit + 1);             // numerator reference less the softmax's [kCW][8]
  float *merge_m = merge_d + C::kCW * 8;                            // softmax reference
  float *merge_l = merge_m + C::kCW * 8;                            // softmax sum
  int *abort_flag = reinterpret_cast<int *>(merge_l + C::kCW * 8);
  const PagedFp8Args &a = p.a;
  const WaitCtx ctx{abort_flag, a.status, wait_limit_ns(a.status)};
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int s = 0; s < C::kStages; ++s) {
      mbar_init(&full[s], 1 + 32 * C::kPW);   // one expect_tx, and every producer lane's scale copies
      mbar_init(&empty[s], C::kCW);
    }
    mbar_init(meet, C::kCW);
    mbar_init(merge_full, C::kCW);
    mbar_init(merge_free, C::kPW);
    for (int i = 0; i < C::kQSlots; ++i) mbar_init(&q_full[i], 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  // (what may overlap the kernel before it ends here: 0.6 us of a short call)
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (!p.whole) asm volatile("griddepcontrol.launch_dependents;");

  if (warp >= C::kCW) {
    // ------------------------------------------------------------- producers
    // One control flow for every producer warp: lane (kv, c) looks after keys
    // 16c .. 16c+15 of K (kv = 0) or V (kv = 1), c in the warp's share; the first
    // warp's lane 0 also writes the stage's description.
    const int pw = warp - C::kCW;
    const bool lead = pw == 0 && lane == 0;
    if (lead) {
      tma_prefetch_desc(&tmK);
      tma_prefetch_desc(&tmV);
    }
    // (short sequences: the first item's length, on its way while the CTA meets)
    const int n_first = p.whole ? a.seqlens[min(static_cast<int>(blockIdx.x) / a.Hkv, a.B - 1)] : 0;
    named_barrier_sync(kBarInit, C::kThreads);      // the barriers are initialised
    const int kv = lane >> 4, c = pw * C::kShare + (lane & 15);
    const int rows = p.box_rows;
    const bool active = (lane & 15) < C::kShare;
    const bool issues = active && (c * 16) % rows == 0;   // this lane's 16 keys start a box
    const uint8_t *scales = kv ? a.vscales : a.kscales;
    const int64_t sc_page = kv ? a.vs_s[0] : a.ks_s[0], sc_head = kv ? a.vs_s[1] : a.ks_s[1];
    const int step = gridDim.x;
    int item = blockIdx.x, items;
    // ---- plan: every producer warp finds the CTA's share for itself (the
    // consumers need none of it).  Lane l counts the tiles of a run of sequences;
    // a scan over the warp gives every run's first tile and the total.
    int E = 0, n_next = n_first;
    long long span = 0, rem = 0;         // spans of span + 1 tiles, rem of them, then of span
    auto span_start = [&](int j) { return j * span + min(static_cast<long long>(j), rem); };
    // the sequence that holds an item's first tile, and its own first tile: where
    // the walk of the items of one span, and of the next, begins
    int b_from = 0;
    long long base_from = 0;
    if (p.whole) {
      items = a.B * a.Hkv;
    } else {
      const int per = (a.B + 31) / 32;
      const int run0 = min(a.B, lane * per), run1 = min(a.B, run0 + per);
      long long mine = 0;
#pragma unroll 4
      for (int b = run0; b < run1; ++b) mine += range_of<C::kTK>(p, a.seqlens[b]).tiles;
      long long incl = mine;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const long long y = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += y;
      }
      const long long total = __shfl_sync(0xffffffffu, incl, 31);
      E = static_cast<int>(min(static_cast<long long>(p.teams), total));   // spans in use
      items = E * a.Hkv;
      if (blockIdx.x == 0 && lead) p.info[p.teams] = make_int2(E, 0);
      if (item < items) {
        span = div_ll(total, E);
        rem = total - span * E;
        const long long first_tile = span_start(item / a.Hkv);
        const uint32_t owner = __ballot_sync(0xffffffffu, incl - mine <= first_tile && first_tile < incl);
        const int src = __ffs(owner) - 1;
        b_from = __shfl_sync(0xffffffffu, run0, src);
        base_from = __shfl_sync(0xffffffffu, incl - mine, src);
      }
    }

    // ---- the pieces, one after another: tiles i .. i1-1 of sequence b (range r),
    // kv head hk, for the partial slot dest (-1: the sequence is finished here)
    int b = 0, hk = 0, i = 0, i1 = 0, i_first = 0, dest = -1, team = 0;
    long long t = 0, t1 = 0, base = 0;
    int note = -1;                       // the sequence that begins in this span and is cut by its end
    long long note_tile = 0;             // and its last tile
    Range r{};
    bool in_item = false;
    auto next_piece = [&]() -> bool {
      if (p.whole) {
        for (; item < items; item += step) {
          b = item / a.Hkv;
          hk = item - b * a.Hkv;
          r = range_of<C::kTK>(p, n_next);
          if (item + step < items) n_next = a.seqlens[(item + step) / a.Hkv];
          if (r.tiles > 0) {
            i = i_first = 0;
            i1 = r.tiles;
            item += step;
            return true;
          }
          for (int e = pw * 32 + lane; e < p.G * D; e += C::kPW * 32)
            a.out[b * a.o_s[0] + (hk * p.G + e / D) * a.o_s[1] + e % D] = __float2bfloat16_rn(0.f);
        }
        return false;
      }
      if (in_item && t >= t1) {          // the item is issued
        if (hk == 0 && lead) {
          const long long wide = rem * (span + 1);    // tiles of the longer spans
          int2 out = make_int2(note, 0);
          if (note >= 0)
            out.y = static_cast<int>(note_tile < wide ? div_ll(note_tile, span + 1) : rem + div_ll(note_tile - wide, span));
          p.info[team] = out;
        }
        in_item = false;
        item += step;
      }
      if (!in_item) {
        if (item >= items) return false;
        team = item / a.Hkv;
        hk = item - team * a.Hkv;
        t = span_start(team);
        t1 = span_start(team + 1);
        b = b_from;
        base = base_from;
        r = range_of<C::kTK>(p, a.seqlens[b]);
        note = -1;
      }
      while (t >= base + r.tiles) {
        base += r.tiles;
        r = range_of<C::kTK>(p, a.seqlens[++b]);
      }
      if (!in_item) {
        b_from = b;
        base_from = base;
        in_item = true;
      }
      i = i_first = static_cast<int>(t - base);
      i1 = static_cast<int>(min(static_cast<long long>(r.tiles), t1 - base));
      if (i == 0 && i1 < r.tiles) {
        note = b;
        note_tile = base + r.tiles - 1;
      }
      dest = i == 0 && i1 == r.tiles ? -1 : 2 * team + (i == 0 ? 1 : 0);
      t = base + i1;
      return true;
    };
    auto page_of = [&](int tile) -> int {   // pool page of this lane's 16 keys of a tile
      const int key = r.start + tile * C::kTK + c * 16;
      if (!active || tile >= i1 || key >= r.n) return -1;
      const int pg = a.block_table[static_cast<int64_t>(b) * a.bt_s0 + (key >> p.page_shift)];
      return pg >= 0 && pg < a.npages ? pg : -1;
    };
    // The last producer warp prepares a piece's q: f16 under a power of two per
    // head that puts its largest magnitude in [2^13, 2^14) (exact for elements
    // above max * 2^-27); k = 2t, 2t+1, 2t+8, 2t+9 of a k-step hold d = 4t .. 4t+3
    // of its 16, the order K's bytes arrive in.  Its loads leave before the piece's
    // first tile is issued, the rest follows it.
    uint32_t qx[NT][D / 16][2];
    auto load_q = [&]() {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        const int hl = nt * 8 + (lane >> 2);
        const __nv_bfloat16 *qr = a.q + b * a.q_s[0] + (hk * p.G + hl) * a.q_s[1] + 4 * (lane & 3);
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          qx[nt][kk][0] = qx[nt][kk][1] = 0u;
          if (hl < p.G) {
            qx[nt][kk][0] = *reinterpret_cast<const uint32_t *>(qr + kk * 16);
            qx[nt][kk][1] = *reinterpret_cast<const uint32_t *>(qr + kk * 16 + 2);
          }
        }
      }
    };
    auto prepare_q = [&](int qs) {
      uint2 *qsm = reinterpret_cast<uint2 *>(smem + C::kQOffset + qs * C::kQSlot) + lane;
      float *qscale = reinterpret_cast<float *>(smem + C::kQOffset + qs * C::kQSlot + C::kQScale);
      float back[NT];                    // 2^-e of this lane's head
      bool large = false;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        float mx = 0.f;
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk)
#pragma unroll
          for (int f = 0; f < 2; ++f)
            mx = fmaxf(mx, fmaxf(fabsf(__uint_as_float(qx[nt][kk][f] << 16)), fabsf(__uint_as_float(qx[nt][kk][f] & 0xFFFF0000u))));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
        // 13 - floor(log2 mx), from the exponent's bits; at most 126, so that the
        // scale itself stays finite (a smaller q only lies lower in f16's range);
        // 0 where the head holds an infinity
        const int eb = static_cast<int>(__float_as_uint(mx) >> 23);
        const int e = eb == 255 ? 0 : min(140 - eb, 126);
        const float sc = __uint_as_float(static_cast<uint32_t>(127 + e) << 23);
        back[nt] = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
        large |= isinf(p.scale_log2 * (1.f / kDown) * back[nt]);
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk)
          qsm[(kk * NT + nt) * 32] = make_uint2(f32x2_to_f16x2(qx[nt][kk][0], sc), f32x2_to_f16x2(qx[nt][kk][1], sc));
      }
      const float down = __any_sync(0xffffffffu, large) ? 1.f : kDown;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
        // (never 0, which would make NaN of a masked key's -infinity)
        if ((lane & 3) == 0)
          qscale[nt * 8 + (lane >> 2)] = fmaxf(p.scale_log2 * (1.f / down) * back[nt], __uint_as_float(1u));
      if (lane == 0) qscale[NT * 8] = down;
      __syncwarp();
      if (lane == 0) mbar_arrive(&q_full[qs]);
    };

    // ---- one loop: issue tiles, then the end mark, then wait for the last merges;
    // before each, merge what the consumers have left meanwhile (one copy of that
    // code: every copy is fetched cold where it first runs)
    int slot = 0, pieces = 0, merged = 0, pg_next = -1, qs = 0;
    enum { kTiles, kMark, kRest };
    int job = kTiles;
    bool ok = true;
    for (;;) {
      if (job == kTiles && i == i1) {
        if (next_piece()) {
          pg_next = page_of(i);
          if (pw == C::kPW - 1) load_q();
        } else {
          job = kMark;
        }
      }
      const int s = slot % C::kStages;
      const uint32_t parity = (static_cast<uint32_t>(slot / C::kStages) & 1u) ^ 1u;
      // Bounded wait for the stage (the last job: for every unit to be merged),
      // merging units meanwhile: the stage may be one that a unit holds.
      uint64_t w0 = 0;
      for (;;) {
        int st = 0;                      // 1 the stage is free, 2 given up, 3 a unit to merge
        if (lane == 0) {
          if (merged < pieces * NT && mbar_test_wait(merge_full, static_cast<uint32_t>(merged) & 1u)) st = 3;
          else if (job == kRest) st = merged == pieces * NT ? 1 : 0;
          else if (slot < C::kStages || mbar_test_wait(&empty[s], parity)) st = 1;
          if (st == 0) {
            if (w0 == 0) {
              w0 = globaltimer_ns();
            } else if (*ctx.abort) {
              st = 2;
            } else if (globaltimer_ns() - w0 > ctx.limit) {
              report_timeout(ctx.status, job == kRest ? kWhereMerge : kWhereEmpty);
              *ctx.abort = 1;
              st = 2;
            } else {
              const uint32_t nap = ctx.limit < 500 ? static_cast<uint32_t>(ctx.limit) : 500u;
              if (job == kRest) mbar_try_wait_sleep(merge_full, static_cast<uint32_t>(merged) & 1u, nap);
              else if (mbar_try_wait_sleep(&empty[s], parity, nap)) st = 1;
            }
          }
        }
        st = __shfl_sync(0xffffffffu, st, 0);
        __syncwarp();
        if (st == 2) ok = false;
        if (st == 1 || st == 2) break;
        if (st == 3) {
          const MergeUnit u = *unit;
          const float *mbuf = reinterpret_cast<const float *>(smem + u.stage * C::kStageBytes);   // [warp][8 heads][D]
          const int heads = min(p.G - u.nt * 8, 8);
          for (int e = pw * 32 + lane; e < heads * (D / 4); e += C::kPW * 32) {
            const int hl = e / (D / 4), d = (e - hl * (D / 4)) * 4;
            const int hq = u.hk * p.G + u.nt * 8 + hl;
            // (first, so that its latency overlaps the sums; the sink joins here if no
            // other span holds keys of this sequence)
            const float sink2 = u.dest < 0 ? a.sinks[hq] * kLog2e : -INFINITY;
            float M = kNoMax;
#pragma unroll
            for (int w = 0; w < C::kCW; ++w) M = fmaxf(M, merge_m[w * 8 + hl]);
            float N = kNoMax, den = 0.f;   // the numerator's reference, less M
#pragma unroll
            for (int w = 0; w < C::kCW; ++w) {
              const float below = merge_m[w * 8 + hl] - M;
              N = fmaxf(N, below + merge_d[w * 8 + hl]);
              den += merge_l[w * 8 + hl] * ex2_approx(below);
            }
            // the numerator on its own largest reference: 2^N joins only behind the
            // division, so that neither the sum of large values nor the weights of small
            // ones leave f32 where their mean does not
            float4 num = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int w = 0; w < C::kCW; ++w) {
              const float f = ex2_approx(merge_m[w * 8 + hl] - M + merge_d[w * 8 + hl] - N);
              const float4 v = *reinterpret_cast<const float4 *>(mbuf + (w * 8 + hl) * D + (d ^ (hl >> 1 << 3)));
              num.x = fmaf(f, v.x, num.x);
              num.y = fmaf(f, v.y, num.y);
              num.z = fmaf(f, v.z, num.z);
              num.w = fmaf(f, v.w, num.w);
            }
            // on the larger of the keys' and the sink's reference: no exponent is positive
            const float M1 = fmaxf(M, sink2), back = ex2_approx(M - M1);
            den = den * back + ex2_approx(sink2 - M1);
            const float inv = den != 0.f ? back / den : 0.f;
            // (in two halves: N goes down to -132)
            const float up = ex2_approx(0.5f * N);
            num = make_float4(num.x * inv * up * up, num.y * inv * up * up, num.z * inv * up * up, num.w * inv * up * up);
            if (u.dest < 0) {
              __nv_bfloat16 *po = a.out + u.b * a.o_s[0] + hq * a.o_s[1] + d;
              if (p.out8) {
                *reinterpret_cast<uint2 *>(po) = make_uint2(pack_bf16x2(num.x, num.y), pack_bf16x2(num.z, num.w));
              } else {
                po[0] = __float2bfloat16_rn(num.x);
                po[1] = __float2bfloat16_rn(num.y);
                po[2] = __float2bfloat16_rn(num.z);
                po[3] = __float2bfloat16_rn(num.w);
              }
            } else {
              const size_t row = static_cast<size_t>(u.dest) * a.Hq + hq;
              *reinterpret_cast<float4 *>(p.o_part + row * D + d) = num;
              if (d == 0) p.lse_part[row] = (M1 + log2f(den)) * kLn2;
            }
          }
          // the generic reads are ordered before the next TMA write into the stage
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) {
            mbar_arrive(merge_free);
            if (u.last) mbar_arrive_n(&empty[u.stage], C::kCW / C::kPW);
          }
          ++merged;
          w0 = 0;
        }
      }
      if (!ok || job == kRest) break;
      ++slot;
      if (job == kMark) {
        if (lead) {
          info[s].flags = 4;
          mbar_arrive(&full[s]);
        }
        __syncwarp();
        copy_async_arrive(&full[s]);
        job = kRest;
        continue;
      }
      // ---- tile i into stage s ----
      const int pg = pg_next;
      pg_next = page_of(i + 1);            // (read a tile ahead: its latency overlaps the next wait)
      const int key0 = r.start + i * C::kTK;
      const int nvalid = min(C::kTK, r.n - key0);
      // only the boxes that hold a valid key are loaded; the rest of the
      // stage keeps old bytes, which are masked
      const int nbox = (nvalid + rows - 1) >> p.box_shift;
      const bool first = i == i_first;
      if (lead) {
        StageInfo &si = info[s];
        si.b = b;
        si.hk = hk;
        si.dest = dest;
        si.nvalid = nvalid;
        si.nskip = max(0, r.vis0 - key0);
        si.flags = (first ? 1 : 0) | (i == i1 - 1 ? 2 : 0);
        mbar_arrive_expect_tx(&full[s], static_cast<uint32_t>(nbox) * rows * D * 2);
      }
      __syncwarp();
      uint8_t *stage = smem + s * C::kStageBytes + kv * C::kTileBytes;
      const int key = key0 + c * 16;
      const int at = key & (a.page - 1);
      // An entry outside the pool reads as a page of zero rows: the box is
      // out of range and filled with zeros (it still delivers its bytes).
      if (issues && c * 16 < nbox * rows)
        tma_load_5d(stage + c * 16 * D, kv ? &tmV : &tmK, &full[s], 0, at, 0, hk, pg);
      if (active && c * 16 < nvalid)
        copy16_async(smem + C::kScaleOffset + s * C::kScaleBytes + kv * C::kTK + c * 16,
                     scales + (pg < 0 ? 0 : pg * sc_page + hk * sc_head + at), pg >= 0);
      copy_async_arrive(&full[s]);
      if (first) {
        if (pw == C::kPW - 1) prepare_q(qs);
        qs = qs + 1 == C::kQSlots ? 0 : qs + 1;
        ++pieces;
      }
      ++i;
    }
    // Every copy has landed before this warp leaves: the CTA's shared memory
    // outlives them, also when the consumers gave up early (each wait is bounded
    // by the fixed limit, whatever limit the other waits use).
    copy_async_wait_all();
    for (int x = max(0, slot - C::kStages); x < slot; ++x) {
      const uint64_t w0 = globaltimer_ns();
      while (!mbar_try_wait(&full[x % C::kStages], static_cast<uint32_t>(x / C::kStages) & 1u))
        if (globaltimer_ns() - w0 > kWaitLimitNs) break;
    }
    __syncwarp();
    return;
  }

  named_barrier_sync(kBarInit, C::kThreads);
  // ------------------------------------------------------------- consumers
  const int g8 = lane >> 2;       // key row within an 8-row block of S^T
  const int tig = lane & 3;       // heads 2*tig, 2*tig+1 of a head tile
  const int key_w = warp * 16 * C::kKB;   // this warp's keys within a tile
  const int bs = p.box_shift;
  // Byte offset of (key row, 16-byte unit u of the row): [box][chunk][row in
  // box][kInner bytes], 128- or 64-byte swizzle.
  const int krow = key_w + (lane & 7) + ((lane >> 3) & 1) * 8;
  const uint32_t row_off =
      D == 256 ? static_cast<uint32_t>((((krow >> bs) * C::kChunks) << (bs + 7)) + ((krow & (p.box_rows - 1)) << 7))
               : static_cast<uint32_t>(krow * C::kInner);
  const uint32_t chunk_stride = 128u << bs;                          // (D = 256)
  const uint32_t swz = D == 64 ? (krow >> 1) & 3 : krow & 7;
  // (block kb is 16 rows on; D = 256 has one block)
  auto unit_off = [&](int u, int kb) -> uint32_t {
    if (D == 256) return row_off + (u >> 3) * chunk_stride + (((u & 7) ^ swz) << 4);
    return row_off + kb * 16 * C::kInner + ((u ^ swz) << 4);
  };
  uint32_t qf[C::kQInSmem ? 1 : D / 16][NT][2];   // B fragments of q^T per k-step and head tile
  int q_off = 0;                                  // where they are in shared memory
  float o[D / 16][NT][4];                         // O^T accumulators: [d tile][head tile][fragment]
  float sl[NT][2];                                // softmax scale of this lane's heads (with q's power of two)
  // softmax reference and numerator reference (less headroom) minus that: one per
  // head, the same in every lane; softmax sum of this lane's keys
  float m_ref[NT][2], d_ref[NT][2], l_run[NT][2];
  int piece = -1, units = 0;
  for (int slot = 0;; ++slot) {
    const int s = slot % C::kStages;
    if (!warp_wait(&full[s], static_cast<uint32_t>(slot / C::kStages) & 1u, ctx, kWhereFull)) break;
    const StageInfo si = info[s];
    if (si.flags & 4) break;
    const uint32_t kbase = smem_u32(smem + s * C::kStageBytes);
    const uint32_t vbase = kbase + C::kTileBytes;
    if (si.flags & 1) {
      // a piece begins: its queries
      ++piece;
      const int qs = piece % C::kQSlots;
      if (!warp_wait(&q_full[qs], static_cast<uint32_t>(piece / C::kQSlots) & 1u, ctx, kWhereFull)) break;
      q_off = C::kQOffset + qs * C::kQSlot;
      const uint2 *qsm = reinterpret_cast<const uint2 *>(smem + q_off) + lane;
      const float *qscale = reinterpret_cast<const float *>(smem + q_off + C::kQScale);
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        sl[nt][0] = qscale[nt * 8 + 2 * tig];
        sl[nt][1] = qscale[nt * 8 + 2 * tig + 1];
#pragma unroll
        for (int f = 0; f < 2; ++f) {
          m_ref[nt][f] = kNoMax;
          d_ref[nt][f] = l_run[nt][f] = 0.f;
        }
        if constexpr (!C::kQInSmem) {
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk) {
            const uint2 f = qsm[(kk * NT + nt) * 32];
            qf[kk][nt][0] = f.x;
            qf[kk][nt][1] = f.y;
          }
        }
      }
#pragma unroll
      for (int dm = 0; dm < D / 16; ++dm)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int f = 0; f < 4; ++f) o[dm][nt][f] = 0.f;
    }
    // a warp none of whose keys is visible has nothing to add
    if (si.nvalid > key_w && si.nskip < key_w + 16 * C::kKB) {
      // all of the warp's keys visible (the common case): nothing is masked
      const bool whole = si.nskip <= key_w && si.nvalid >= key_w + 16 * C::kKB;
      // ---- S^T[16 keys x 8*NT heads] = K_w q^T, per key block ----
      // (two chains of accumulators where there would be one: the products of a
      // chain wait for one another)
      constexpr int KB = C::kKB;
      constexpr int kChains = NT * KB == 1 ? 2 : 1;
      float sacc[KB][kChains][NT][4];
#pragma unroll
      for (int kb = 0; kb < KB; ++kb)
#pragma unroll
        for (int ch = 0; ch < kChains; ++ch)
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int f = 0; f < 4; ++f) sacc[kb][ch][nt][f] = 0.f;
#pragma unroll
      for (int up = 0; up < D / 32; ++up)
#pragma unroll
        for (int kb = 0; kb < KB; ++kb) {
          // matrices (keys 0-7 | 8-15) x (16-byte unit u | u+1): lane (g, t)
          // receives d = 16u + 4t .. 4t+3 of keys g and g + 8
          uint32_t w0, w1, w2, w3;
          ldmatrix_x4(kbase + unit_off(2 * up + (lane >> 4), kb), w0, w1, w2, w3);
          const uint2 k0 = e4m3x4_to_f16x2x2(w0), k1 = e4m3x4_to_f16x2x2(w1);
          const uint2 k2 = e4m3x4_to_f16x2x2(w2), k3 = e4m3x4_to_f16x2x2(w3);
          const int kk = 2 * up;
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            uint2 qa, qb;
            if constexpr (C::kQInSmem) {
              const uint2 *qsm = reinterpret_cast<const uint2 *>(smem + q_off) + lane;
              qa = qsm[(kk * NT + nt) * 32];
              qb = qsm[((kk + 1) * NT + nt) * 32];
            } else {
              qa = make_uint2(qf[kk][nt][0], qf[kk][nt][1]);
              qb = make_uint2(qf[kk + 1][nt][0], qf[kk + 1][nt][1]);
            }
            mma_f16_16816(sacc[kb][0][nt], k0.x, k1.x, k0.y, k1.y, qa.x, qa.y);
            mma_f16_16816(sacc[kb][kChains - 1][nt], k2.x, k3.x, k2.y, k3.y, qb.x, qb.y);
          }
        }
      // ---- softmax terms (no sink here) ----
      // t = S * kscale; the softmax's exponent is t * sl - M, one FMA, the numerator's
      // lies ev - (m - M) above it: m is held as its distance from M, so that logits
      // too large for their difference of a few binades do not lose it.
      float t[KB][NT][4], ev[KB][2];
      const float down = *reinterpret_cast<const float *>(smem + q_off + C::kQScale + NT * 8 * 4);
#pragma unroll
      for (int kb = 0; kb < KB; ++kb) {
        const uint8_t *sck = smem + C::kScaleOffset + s * C::kScaleBytes + key_w + kb * 16 + g8;
        float ks[2];
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          const uint32_t b = sck[r * 8], vb = sck[C::kTK + r * 8];
          ks[r] = scale_value(b) * down;
          // vb - 127 by way of 2^23 + vb, exact
          ev[kb][r] = vb == 255u ? NAN : __uint_as_float(0x4B000000u | vb) - 8388735.f;
        }
        if constexpr (kChains == 2) {
#pragma unroll
          for (int f = 0; f < 4; ++f) sacc[kb][0][0][f] += sacc[kb][1][0][f];
        }
        if (!whole) {
          const int i0 = key_w + kb * 16 + g8;
#pragma unroll
          for (int r = 0; r < 2; ++r)
            if (i0 + r * 8 < si.nskip || i0 + r * 8 >= si.nvalid) {
#pragma unroll
              for (int nt = 0; nt < NT; ++nt) sacc[kb][0][nt][2 * r] = sacc[kb][0][nt][2 * r + 1] = -INFINITY;
              ks[r] = 1.f;
              ev[kb][r] = 0.f;
            }
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int f = 0; f < 4; ++f) t[kb][nt][f] = sacc[kb][0][nt][f] * ks[f >> 1];   // key g + 8*(f>>1), head 2*tig + (f&1)
      }
      float zd[KB][NT][4], zn[KB][NT][4];
      auto exponents = [&]() {
#pragma unroll
        for (int kb = 0; kb < KB; ++kb)
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int f = 0; f < 4; ++f) {
              zd[kb][nt][f] = fmaf(t[kb][nt][f], sl[nt][f & 1], -m_ref[nt][f & 1]);
              zn[kb][nt][f] = zd[kb][nt][f] + (ev[kb][f >> 1] - d_ref[nt][f & 1]);
            }
      };
      exponents();
      float top_d = -INFINITY, top_n = -INFINITY;
#pragma unroll
      for (int kb = 0; kb < KB; ++kb)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int f = 0; f < 4; f += 2) {
            top_d = fmaxf(top_d, fmaxf(zd[kb][nt][f], zd[kb][nt][f + 1]));
            top_n = fmaxf(top_n, fmaxf(zn[kb][nt][f], zn[kb][nt][f + 1]));
          }
      if (__any_sync(0xffffffffu, top_d > kLazy || top_n > kLazy + kHeadroom)) {
        // a reference is left behind (always on a piece's first tile, rarely
        // after it): move both up to the maxima seen
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int f = 0; f < 2; ++f) {
            float m1 = -INFINITY, d1 = -INFINITY;
#pragma unroll
            for (int kb = 0; kb < KB; ++kb)
              m1 = fmaxf(m1, fmaxf(t[kb][nt][f] * sl[nt][f], t[kb][nt][f + 2] * sl[nt][f]));
#pragma unroll
            for (int off = 4; off < 32; off <<= 1) m1 = fmaxf(m1, __shfl_xor_sync(0xffffffffu, m1, off));
            m1 = fmaxf(m_ref[nt][f], m1);
            const float fall = m_ref[nt][f] - m1;
            l_run[nt][f] *= ex2_approx(fall);
            m_ref[nt][f] = m1;
#pragma unroll
            for (int kb = 0; kb < KB; ++kb)
              d1 = fmaxf(d1, fmaxf(fmaf(t[kb][nt][f], sl[nt][f], -m1) + ev[kb][0],
                                   fmaf(t[kb][nt][f + 2], sl[nt][f], -m1) + ev[kb][1]));
#pragma unroll
            for (int off = 4; off < 32; off <<= 1) d1 = fmaxf(d1, __shfl_xor_sync(0xffffffffu, d1, off));
            const float d0 = d_ref[nt][f] + fall;
            d1 = fmaxf(d0, d1 - kHeadroom);
            const float al = ex2_approx(d0 - d1);
            d_ref[nt][f] = d1;
#pragma unroll
            for (int dm = 0; dm < D / 16; ++dm) {
              o[dm][nt][f] *= al;
              o[dm][nt][f + 2] *= al;
            }
          }
        exponents();
      }
      uint32_t pb[KB][NT][2];
#pragma unroll
      for (int kb = 0; kb < KB; ++kb)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          const float *d = zd[kb][nt], *n = zn[kb][nt];
          l_run[nt][0] += ex2_approx(d[0]) + ex2_approx(d[2]);
          l_run[nt][1] += ex2_approx(d[1]) + ex2_approx(d[3]);
          // P^T fragments, transposed into the B operand of O^T += V^T P^T
          pb[kb][nt][0] = movmatrix_trans(pack_f16x2(ex2_approx(n[0]), ex2_approx(n[1])));
          pb[kb][nt][1] = movmatrix_trans(pack_f16x2(ex2_approx(n[2]), ex2_approx(n[3])));
        }
      // ---- O^T[D x 8*NT] += V_w^T P^T ----
      // ldmatrix.trans of bytes taken as 16-bit pairs: lane (g, t) receives
      // keys 2t, 2t+1 (2t+8, 2t+9) at d = 16u + 2g and 2g + 1; one byte permute
      // makes key pairs per d, so O^T rows g and g + 8 of d tile u are d = 16u +
      // 2g and 16u + 2g + 1.  Codes of keys outside [nskip, nvalid) may be
      // anything (NaN included): on the tiles that have any they are zeroed here.
      auto pv = [&](auto masked) {
#pragma unroll
        for (int kb = 0; kb < KB; ++kb) {
          uint32_t blo = 0xFFFFFFFFu, bhi = 0xFFFFFFFFu;   // bytes: keys k, k+1 of d even, then of d odd
          if constexpr (decltype(masked)::value) {
            const int ka = key_w + kb * 16 + 2 * tig;
            auto in = [&](int k) { return k >= si.nskip && k < si.nvalid; };
            blo = (in(ka) ? 0x00FF00FFu : 0u) | (in(ka + 1) ? 0xFF00FF00u : 0u);
            bhi = (in(ka + 8) ? 0x00FF00FFu : 0u) | (in(ka + 9) ? 0xFF00FF00u : 0u);
          }
#pragma unroll
          for (int up = 0; up < D / 32; ++up) {
            uint32_t w0, w1, w2, w3;
            ldmatrix_x4_trans(vbase + unit_off(2 * up + (lane >> 4), kb), w0, w1, w2, w3);
            w0 = __byte_perm(w0, 0u, 0x3120);
            w1 = __byte_perm(w1, 0u, 0x3120);
            w2 = __byte_perm(w2, 0u, 0x3120);
            w3 = __byte_perm(w3, 0u, 0x3120);
            if constexpr (decltype(masked)::value) {
              w0 &= blo;
              w1 &= bhi;
              w2 &= blo;
              w3 &= bhi;
            }
            const uint2 v0 = e4m3x4_to_f16x2x2(w0), v1 = e4m3x4_to_f16x2x2(w1);
            const uint2 v2 = e4m3x4_to_f16x2x2(w2), v3 = e4m3x4_to_f16x2x2(w3);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              mma_f16_16816(o[2 * up][nt], v0.x, v0.y, v1.x, v1.y, pb[kb][nt][0], pb[kb][nt][1]);
              mma_f16_16816(o[2 * up + 1][nt], v2.x, v2.y, v3.x, v3.y, pb[kb][nt][0], pb[kb][nt][1]);
            }
          }
        }
      };
      if (whole)
        pv(std::false_type{});
      else
        pv(std::true_type{});
    }
    // the stage is only read here: release it, but the last one of a piece only
    // after the merge that reuses its memory
    if (!(si.flags & 2)) {
      __syncwarp();
      if (lane == 0) mbar_arrive(&empty[s]);
      continue;
    }
    // ---- a piece ends: leave the warp's state in the stage ----
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int f = 0; f < 2; ++f) {
#pragma unroll
        for (int off = 4; off < 32; off <<= 1) l_run[nt][f] += __shfl_xor_sync(0xffffffffu, l_run[nt][f], off);
      }
    // every warp is done with this stage
    __syncwarp();
    if (lane == 0) mbar_arrive(meet);
    if (!warp_wait(meet, static_cast<uint32_t>(piece) & 1u, ctx, kWhereMerge)) break;
    float *mw = reinterpret_cast<float *>(smem + s * C::kStageBytes) + warp * 8 * D;   // [warp][8 heads][D]
    bool left = false;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      // the previous unit has been read
      if (units > 0 && !warp_wait(merge_free, static_cast<uint32_t>(units - 1) & 1u, ctx, kWhereMerge)) {
        left = true;
        break;
      }
      if (g8 == 0) {
#pragma unroll
        for (int f = 0; f < 2; ++f) {
          const int at = warp * 8 + 2 * tig + f;
          merge_d[at] = d_ref[nt][f];
          merge_m[at] = m_ref[nt][f];
          merge_l[at] = l_run[nt][f];
        }
      }
#pragma unroll
      for (int dm = 0; dm < D / 16; ++dm) {
        // (the head pairs of a store's lanes go to different banks)
        const int d = (dm * 16 + 2 * g8) ^ (tig << 3);
        *reinterpret_cast<float2 *>(mw + 2 * tig * D + d) = make_float2(o[dm][nt][0], o[dm][nt][2]);
        *reinterpret_cast<float2 *>(mw + (2 * tig + 1) * D + d) = make_float2(o[dm][nt][1], o[dm][nt][3]);
      }
      if (warp == 0 && lane == 0) *unit = MergeUnit{si.b, si.hk, si.dest, nt, s, nt == NT - 1, 0, 0};
      // (ordered before the next TMA write into the stage)
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(merge_full);
      ++units;
    }
    if (left) break;
  }
}

// ---------------------------------------------------------------- combine
// One warp per (span that begins a cut sequence, query head), then one warp per
// 32 sequences to write the rows of the empty ones.
template <int D>
__global__ void __launch_bounds__(128) paged_fp8_combine_kernel(const __grid_constant__ Params p) {
  constexpr int kPer = D / 32;                      // channels per lane, consecutive
  constexpr int kAhead = 4;                         // parts whose loads do not wait for the weights
  const PagedFp8Args &a = p.a;
  const int lane = threadIdx.x & 31;
  const long long w = (static_cast<long long>(blockIdx.x) * blockDim.x + threadIdx.x) >> 5;
  const long long merges = static_cast<long long>(p.teams) * a.Hq;
  if (w >= merges) {
    const long long b0 = (w - merges) * 32;
    if (b0 >= a.B) return;
    const int n = b0 + lane < a.B ? min(a.seqlens[b0 + lane], a.max_pages << p.page_shift) : 1;
    uint32_t empty = __ballot_sync(0xffffffffu, n <= 0);
    while (empty) {
      const long long b = b0 + __ffs(empty) - 1;
      empty &= empty - 1;
      for (int e = lane; e < a.Hq * D; e += 32) a.out[b * a.o_s[0] + (e / D) * a.o_s[1] + e % D] = __float2bfloat16_rn(0.f);
    }
    return;
  }
  const int team = static_cast<int>(w / a.Hq), hq = static_cast<int>(w - static_cast<long long>(team) * a.Hq);
  const float sink = a.sinks[hq];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int2 note = p.info[team];
  const int E = min(p.info[p.teams].x, p.teams);
  // (checked whole: a split whose waits ran out may not have written its note)
  if (team >= E || note.x < 0 || note.x >= a.B || note.y <= team || note.y >= E) return;
  const int parts = note.y - team + 1;
  // part 0 is the span's own last piece, part i the first piece of span team + i
  auto slot_of = [&](int i) { return static_cast<size_t>(i == 0 ? 2 * team + 1 : 2 * (team + i)) * a.Hq + hq; };
  float ahead[kAhead][kPer];
#pragma unroll
  for (int i = 0; i < kAhead; ++i)
#pragma unroll
    for (int t = 0; t < kPer; t += 2) {
      const float2 v = i < parts ? *reinterpret_cast<const float2 *>(p.o_part + slot_of(i) * D + lane * kPer + t)
                                 : make_float2(0.f, 0.f);
      ahead[i][t] = v.x;
      ahead[i][t + 1] = v.y;
    }
  float M = sink;
  for (int i0 = 0; i0 < parts; i0 += 32) {
    float ls = i0 + lane < parts ? p.lse_part[slot_of(i0 + lane)] : -INFINITY;
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) ls = fmaxf(ls, __shfl_xor_sync(0xffffffffu, ls, off));
    M = fmaxf(M, ls);
  }
  const float Mu = M == -INFINITY ? 0.f : M;
  float den = __expf(sink - Mu), wt0 = 0.f;          // wt0: this lane's weight of the first 32 spans
  for (int i0 = 0; i0 < parts; i0 += 32) {
    float wt = i0 + lane < parts ? __expf(p.lse_part[slot_of(i0 + lane)] - Mu) : 0.f;
    if (i0 == 0) wt0 = wt;
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) wt += __shfl_xor_sync(0xffffffffu, wt, off);
    den += wt;
  }
  // (divided before the sum: the spans' means may be as large as f32 holds)
  const float inv = den != 0.f ? 1.f / den : 0.f;
  float acc[kPer];
#pragma unroll
  for (int t = 0; t < kPer; ++t) acc[t] = 0.f;
  for (int i0 = 0; i0 < parts; i0 += 32) {
    const float wt =
        inv * (i0 == 0 ? wt0 : i0 + lane < parts ? __expf(p.lse_part[slot_of(i0 + lane)] - Mu) : 0.f);
    const int cnt = min(32, parts - i0);
    int i = 0;
    if (i0 == 0) {
#pragma unroll
      for (; i < kAhead; ++i) {                  // spans in order
        const float ws = __shfl_sync(0xffffffffu, wt, i);
#pragma unroll
        for (int t = 0; t < kPer; ++t) acc[t] = fmaf(ws, ahead[i][t], acc[t]);
      }
    }
#pragma unroll 4
    for (; i < cnt; ++i) {
      const float ws = __shfl_sync(0xffffffffu, wt, i);
      const float *op = p.o_part + slot_of(i0 + i) * D + lane * kPer;
#pragma unroll
      for (int t = 0; t < kPer; ++t) acc[t] = fmaf(ws, op[t], acc[t]);
    }
  }
  __nv_bfloat16 *po = a.out + static_cast<int64_t>(note.x) * a.o_s[0] + hq * a.o_s[1] + lane * kPer;
#pragma unroll
  for (int t = 0; t < kPer; ++t) po[t] = __float2bfloat16_rn(acc[t]);
}

template <int D, int NT>
cudaError_t launch(const Params &p, int sms, cudaStream_t stream) {
  using C = Cfg<D, NT>;
  const PagedFp8Args &a = p.a;
  alignas(64) CUtensorMap mk, mv;
  cudaError_t e;
  if ((e = make_tma_pages8(&mk, a.kpages, a.npages, a.page, a.Hkv, D, a.kp_s, p.box_rows)) != cudaSuccess) return e;
  if ((e = make_tma_pages8(&mv, a.vpages, a.npages, a.page, a.Hkv, D, a.vp_s, p.box_rows)) != cudaSuccess) return e;
  auto split = paged_fp8_split_kernel<D, NT>;
  if ((e = cudaFuncSetAttribute(split, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmemBytes)) != cudaSuccess)
    return e;
  const int64_t items = p.whole ? static_cast<int64_t>(a.B) * a.Hkv : static_cast<int64_t>(p.teams) * a.Hkv;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(items < sms ? items : sms));
  cfg.blockDim = dim3(C::kThreads);
  cfg.dynamicSmemBytes = C::kSmemBytes;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if ((e = cudaLaunchKernelEx(&cfg, split, mk, mv, p)) != cudaSuccess || p.whole) return e;
  const int64_t warps = static_cast<int64_t>(p.teams) * a.Hq + (a.B + 31) / 32;
  cfg.gridDim = dim3(static_cast<unsigned>((warps + 3) / 4));
  cfg.blockDim = dim3(128);
  cfg.dynamicSmemBytes = 0;
  return cudaLaunchKernelEx(&cfg, paged_fp8_combine_kernel<D>, p);
}

}  // namespace

size_t paged_fp8_workspace_bytes(const PagedFp8Args &a, int sms) {
  return takes_whole(a) ? 0 : layout(a, max_teams(a.Hkv, sms)).total;
}

cudaError_t launch_decode_paged_fp8(const PagedFp8Args &a, void *workspace, int sms, cudaStream_t stream) {
  Params p;
  p.a = a;
  p.G = a.Hq / a.Hkv;
  p.teams = max_teams(a.Hkv, sms);
  p.page_shift = 0;
  while ((1 << p.page_shift) < a.page) ++p.page_shift;
  p.box_rows = a.page < 64 ? a.page : 64;
  p.box_shift = p.page_shift < 6 ? p.page_shift : 6;
  p.out8 = (reinterpret_cast<uintptr_t>(a.out) | (a.o_s[0] * 2) | (a.o_s[1] * 2)) % 8 == 0;
  p.scale_log2 = static_cast<float>(static_cast<double>(a.scale) * 1.4426950408889634);
  p.whole = takes_whole(a);
  p.info = nullptr;
  p.lse_part = p.o_part = nullptr;
  if (!p.whole) {
    const Workspace w = layout(a, p.teams);
    uint8_t *ws = static_cast<uint8_t *>(workspace);
    p.info = reinterpret_cast<int2 *>(ws + w.off_info);
    p.lse_part = reinterpret_cast<float *>(ws + w.off_lse);
    p.o_part = reinterpret_cast<float *>(ws + w.off_o);
  }
  switch (a.D) {
    case 64: return p.G <= 8 ? launch<64, 1>(p, sms, stream) : launch<64, 2>(p, sms, stream);
    case 128: return p.G <= 8 ? launch<128, 1>(p, sms, stream) : launch<128, 2>(p, sms, stream);
    case 256: return p.G <= 8 ? launch<256, 1>(p, sms, stream) : cudaErrorInvalidValue;
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace attnsink
