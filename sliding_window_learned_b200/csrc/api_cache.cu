// api_cache.cu -- the C ABI of the 8-bit paged cache (declared in
// include/attnsink.h): attn_sink_cache_append_fp8, attn_sink_cache_read_fp8,
// attn_sink_decode_paged_fp8, and of attn_sink_fwd_extend, which continues a
// prompt from rows read back.  Argument checks and launches only.
#include <cuda_runtime.h>

#include "../../include/attnsink.h"
#include "api_internal.h"
#include "kernels.h"

namespace attnsink {
namespace {

// What the three calls share: the pools, their scales and the block table.
struct Pools {
  int64_t NB, P, Hkv, D, MP;
  int shift;
};

int check_pools(const attn_tensor *kpages, const attn_tensor *vpages, const attn_tensor *kscales,
                const attn_tensor *vscales, const attn_tensor *block_table, const attn_tensor *seqlens, Pools *o) {
  int rc;
  if ((rc = check_tensor(kpages, "kpages", ATTN_DTYPE_E4M3, 4, true))) return rc;
  o->P = kpages->shape[1];
  o->D = kpages->shape[3];
  if (o->P < 16 || o->P > 65536 || (o->P & (o->P - 1)))
    return fail(ATTN_EUNSUPPORTED, "page size %lld must be a power of two in [16, 65536]", (long long)o->P);
  if (o->D != 64 && o->D != 128 && o->D != 256)
    return fail(ATTN_EUNSUPPORTED, "head dim %lld not supported (64, 128, 256)", (long long)o->D);
  if ((rc = check_tensor(vpages, "vpages", ATTN_DTYPE_E4M3, 4, true))) return rc;
  if ((rc = check_tensor(kscales, "kscales", ATTN_DTYPE_E8M0, 3, true))) return rc;
  if ((rc = check_tensor(vscales, "vscales", ATTN_DTYPE_E8M0, 3, true))) return rc;
  if ((rc = check_tensor(block_table, "block_table", ATTN_DTYPE_I32, 2, false))) return rc;
  if ((rc = check_tensor(seqlens, "seqlens", ATTN_DTYPE_I32, 1, false))) return rc;
  o->NB = kpages->shape[0];
  o->Hkv = kpages->shape[2];
  o->MP = block_table->shape[1];
  for (int d = 0; d < 4; ++d)
    if (vpages->shape[d] != kpages->shape[d]) return fail(ATTN_EINVAL, "vpages shape does not match kpages");
  if (kscales->shape[0] != o->NB || kscales->shape[1] != o->Hkv || kscales->shape[2] != o->P)
    return fail(ATTN_EINVAL, "kscales must be [NB, Hkv, P] = [%lld, %lld, %lld]", (long long)o->NB,
                (long long)o->Hkv, (long long)o->P);
  for (int d = 0; d < 3; ++d)
    if (vscales->shape[d] != kscales->shape[d]) return fail(ATTN_EINVAL, "vscales shape does not match kscales");
  if (o->NB < 1 || o->Hkv < 1) return fail(ATTN_EINVAL, "the pools need at least one page and one kv head");
  if (block_table->shape[0] != seqlens->shape[0]) return fail(ATTN_EINVAL, "block_table and seqlens must have B rows");
  if (seqlens->shape[0] > 1 && seqlens->stride[0] != 1) return fail(ATTN_EINVAL, "seqlens must be contiguous");
  if (seqlens->shape[0] > (1 << 20) || o->NB > (1LL << 31) - 1 || o->MP > (1LL << 30) || o->MP * o->P > (1LL << 30) ||
      o->Hkv > 16384)
    return fail(ATTN_EUNSUPPORTED, "B, Hkv, the pool or pages per sequence * page size too large");
  o->shift = 0;
  while ((1LL << o->shift) < o->P) ++o->shift;
  return ATTN_OK;
}

int cache_call(const attn_tensor *k, const attn_tensor *v, const attn_tensor *kpages, const attn_tensor *vpages,
               const attn_tensor *kscales, const attn_tensor *vscales, const attn_tensor *block_table,
               const attn_tensor *seqlens, const attn_tensor *cu_seqlens, bool append, void *stream,
               const char *name) {
  Pools o;
  int rc = check_pools(kpages, vpages, kscales, vscales, block_table, seqlens, &o);
  if (rc) return rc;
  if ((rc = check_tensor(k, "k", ATTN_DTYPE_BF16, 3, true))) return rc;
  if ((rc = check_tensor(v, "v", ATTN_DTYPE_BF16, 3, true))) return rc;
  if ((rc = check_tensor(cu_seqlens, "cu_seqlens", ATTN_DTYPE_I32, 1, false))) return rc;
  const int64_t T = k->shape[0], B = seqlens->shape[0];
  if (k->shape[1] != o.Hkv || k->shape[2] != o.D)
    return fail(ATTN_EINVAL, "k must be [T, Hkv, D] = [T, %lld, %lld]", (long long)o.Hkv, (long long)o.D);
  for (int d = 0; d < 3; ++d)
    if (v->shape[d] != k->shape[d]) return fail(ATTN_EINVAL, "v shape does not match k");
  if (cu_seqlens->shape[0] != B + 1) return fail(ATTN_EINVAL, "cu_seqlens must have B + 1 = %lld entries", (long long)B + 1);
  if (B > 0 && cu_seqlens->stride[0] != 1) return fail(ATTN_EINVAL, "cu_seqlens must be contiguous");
  if (T > (1LL << 30) || T * o.Hkv > (1LL << 36)) return fail(ATTN_EUNSUPPORTED, "T must be <= 2^30 and T * Hkv <= 2^36");
  if (T == 0 || B == 0) return ATTN_OK;
  CacheArgs a;
  if (append) {
    a.k = static_cast<const __nv_bfloat16 *>(k->data);
    a.v = static_cast<const __nv_bfloat16 *>(v->data);
  } else {
    a.k_out = static_cast<__nv_bfloat16 *>(k->data);
    a.v_out = static_cast<__nv_bfloat16 *>(v->data);
  }
  for (int d = 0; d < 2; ++d) {
    a.k_s[d] = k->stride[d];
    a.v_s[d] = v->stride[d];
    a.ks_s[d] = kscales->stride[d];
    a.vs_s[d] = vscales->stride[d];
  }
  for (int d = 0; d < 3; ++d) {
    a.kp_s[d] = kpages->stride[d];
    a.vp_s[d] = vpages->stride[d];
  }
  a.kpages = static_cast<uint8_t *>(kpages->data);
  a.vpages = static_cast<uint8_t *>(vpages->data);
  a.kscales = static_cast<uint8_t *>(kscales->data);
  a.vscales = static_cast<uint8_t *>(vscales->data);
  a.block_table = static_cast<const int *>(block_table->data);
  a.seqlens = static_cast<const int *>(seqlens->data);
  a.cu_seqlens = static_cast<const int *>(cu_seqlens->data);
  a.bt_s0 = block_table->stride[0];
  a.T = T;
  a.B = static_cast<int>(B);
  a.Hkv = static_cast<int>(o.Hkv);
  a.D = static_cast<int>(o.D);
  a.page_shift = o.shift;
  a.npages = static_cast<int>(o.NB);
  a.max_pages = static_cast<int>(o.MP);
  int sms;
  if ((rc = sm_count(&sms))) return rc;
  const cudaError_t e = launch_cache(a, append, sms, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? ATTN_OK : fail_cuda(e, name);
}

int extend_call(const attn_tensor *q, const attn_tensor *k, const attn_tensor *v, const attn_tensor *cu_seqlens_q,
                const attn_tensor *cu_seqlens_k, int32_t max_seqlen_q, const attn_tensor *sinks, int32_t window,
                float scale, int32_t terms, attn_tensor *out, attn_tensor *lse, void *stream) {
  int rc;
  if ((rc = check_tensor(q, "q", ATTN_DTYPE_BF16, 3, true))) return rc;
  if ((rc = check_tensor(k, "k", ATTN_DTYPE_BF16, 3, true))) return rc;
  if ((rc = check_tensor(v, "v", ATTN_DTYPE_BF16, 3, true))) return rc;
  if ((rc = check_tensor(cu_seqlens_q, "cu_seqlens_q", ATTN_DTYPE_I32, 1, false))) return rc;
  if ((rc = check_tensor(cu_seqlens_k, "cu_seqlens_k", ATTN_DTYPE_I32, 1, false))) return rc;
  if ((rc = check_tensor(sinks, "sinks", ATTN_DTYPE_F32, 1, false))) return rc;
  if ((rc = check_tensor(out, "out", ATTN_DTYPE_BF16, 3, true))) return rc;
  const int64_t T = q->shape[0], Hq = q->shape[1], D = q->shape[2], Tk = k->shape[0], Hkv = k->shape[1];
  if (k->shape[2] != D) return fail(ATTN_EINVAL, "k head dim does not match q");
  for (int d = 0; d < 3; ++d) {
    if (v->shape[d] != k->shape[d]) return fail(ATTN_EINVAL, "v shape does not match k");
    if (out->shape[d] != q->shape[d]) return fail(ATTN_EINVAL, "out shape does not match q");
  }
  const int64_t B = cu_seqlens_q->shape[0] - 1;
  if (B < 0 || cu_seqlens_k->shape[0] != B + 1)
    return fail(ATTN_EINVAL, "cu_seqlens_q and cu_seqlens_k need B + 1 >= 1 entries each");
  if (B > 0 && (cu_seqlens_q->stride[0] != 1 || cu_seqlens_k->stride[0] != 1))
    return fail(ATTN_EINVAL, "cu_seqlens_q and cu_seqlens_k must be contiguous");
  if (sinks->shape[0] != Hq) return fail(ATTN_EINVAL, "sinks must have Hq = %lld entries", (long long)Hq);
  if (Hq > 1 && sinks->stride[0] != 1) return fail(ATTN_EINVAL, "sinks must be contiguous");
  if (Hq <= 0 || Hkv <= 0 || Hq % Hkv) return fail(ATTN_EINVAL, "Hq must be a positive multiple of Hkv");
  if (window < 1) return fail(ATTN_EINVAL, "window must be >= 1");
  if (max_seqlen_q < 0) return fail(ATTN_EINVAL, "max_seqlen_q must be >= 0");
  if (!finite_pos(scale)) return fail(ATTN_EINVAL, "scale must be finite and > 0");
  if (terms < 0 || terms > 2) return fail(ATTN_EINVAL, "terms must be 0, 1 or 2");
  if (lse) {
    if ((rc = check_tensor(lse, "lse", ATTN_DTYPE_F32, 2, false))) return rc;
    if (lse->shape[0] != Hq || lse->shape[1] != T) return fail(ATTN_EINVAL, "lse must be [Hq, T]");
  }
  if (D != 64 && D != 128 && D != 256)
    return fail(ATTN_EUNSUPPORTED, "head dim %lld not supported (64, 128, 256)", (long long)D);
  if (B > 65535 || Hq > 65535 || T > (1LL << 30) || Tk > (1LL << 30))
    return fail(ATTN_EUNSUPPORTED, "B and Hq must be <= 65535, T and Tk <= 2^30");
  // no chunk is longer than T
  const int64_t rows = max_seqlen_q < T ? max_seqlen_q : T;
  // query tiles hold at least 112 rows (position, head) each, but for a sequence's last
  if ((rows * Hq / 112 + Hq) * B > 0x7FFFFFFF)
    return fail(ATTN_EUNSUPPORTED, "(max_seqlen_q / 112 + 1) * Hq * B must be < 2^31");
  if (B == 0 || rows == 0) return ATTN_OK;
  FwdArgs a;
  a.q = q->data;
  a.k = k->data;
  a.v = v->data;
  a.sinks = static_cast<const float *>(sinks->data);
  a.out = out->data;
  a.lse = lse ? static_cast<float *>(lse->data) : nullptr;
  a.B = static_cast<int>(B);
  a.L = static_cast<int>(rows);
  a.T = static_cast<int>(T);
  a.Tk = static_cast<int>(Tk);
  a.Hq = static_cast<int>(Hq);
  a.Hkv = static_cast<int>(Hkv);
  a.D = static_cast<int>(D);
  a.W = window < (1 << 30) ? window : (1 << 30);   // (positions are at least -2^30: no overflow)
  a.scale = scale;
  a.terms = terms;
  a.cu_seqlens = static_cast<const int *>(cu_seqlens_q->data);
  a.cu_seqlens_k = static_cast<const int *>(cu_seqlens_k->data);
  // one batch slice of rows each: its (unused) batch stride spans the slice
  const attn_tensor *ts[4] = {q, k, v, out};
  int64_t *ss[4] = {a.q_s, a.k_s, a.v_s, a.o_s};
  for (int x = 0; x < 4; ++x) {
    ss[x][0] = (ts[x]->shape[0] > 0 ? ts[x]->shape[0] : 1) * ts[x]->stride[0];
    ss[x][1] = ts[x]->stride[0];
    ss[x][2] = ts[x]->stride[1];
  }
  a.lse_s[0] = 0;
  a.lse_s[1] = lse ? lse->stride[0] : 0;
  if ((rc = status_ptr(&a.status))) return rc;
  if ((rc = sm_count(&a.sms))) return rc;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const size_t bytes = fwd_extend_workspace_bytes(a);
  if (bytes == 0) {
    const cudaError_t e = launch_fwd_tc(a, st);
    return e == cudaSuccess ? ATTN_OK : fail_cuda(e, "attn_sink_fwd_extend launch");
  }
  cudaMemPool_t pool;
  if ((rc = workspace_pool(&pool))) return rc;
  if (take_injected_alloc_failure()) return fail(ATTN_ENOMEM, "extend workspace allocation failed (injected)");
  cudaError_t e = cudaMallocFromPoolAsync(&a.workspace, bytes, pool, st);
  if (e != cudaSuccess) return fail_cuda(e, "extend workspace allocation");
  e = launch_fwd_tc(a, st);
  const cudaError_t ef = cudaFreeAsync(a.workspace, st);
  if (e != cudaSuccess) return fail_cuda(e, "attn_sink_fwd_extend launch");
  if (ef != cudaSuccess) return fail_cuda(ef, "extend workspace release");
  return ATTN_OK;
}

}  // namespace
}  // namespace attnsink

using namespace attnsink;

extern "C" {

int attn_sink_cache_append_fp8(const attn_tensor *k, const attn_tensor *v, const attn_tensor *block_table,
                               const attn_tensor *seqlens, const attn_tensor *cu_seqlens, attn_tensor *kpages,
                               attn_tensor *vpages, attn_tensor *kscales, attn_tensor *vscales, void *stream) {
  clear_error();
  return cache_call(k, v, kpages, vpages, kscales, vscales, block_table, seqlens, cu_seqlens, true, stream,
                    "attn_sink_cache_append_fp8 launch");
}

int attn_sink_cache_read_fp8(const attn_tensor *kpages, const attn_tensor *vpages, const attn_tensor *kscales,
                             const attn_tensor *vscales, const attn_tensor *block_table, const attn_tensor *seqlens,
                             const attn_tensor *cu_seqlens, attn_tensor *k, attn_tensor *v, void *stream) {
  clear_error();
  return cache_call(k, v, kpages, vpages, kscales, vscales, block_table, seqlens, cu_seqlens, false, stream,
                    "attn_sink_cache_read_fp8 launch");
}

int attn_sink_decode_paged_fp8(const attn_tensor *q, const attn_tensor *kpages, const attn_tensor *vpages,
                               const attn_tensor *kscales, const attn_tensor *vscales, const attn_tensor *block_table,
                               const attn_tensor *seqlens, const attn_tensor *sinks, int32_t window, float scale,
                               attn_tensor *out, void *stream) {
  clear_error();
  Pools o;
  int rc = check_pools(kpages, vpages, kscales, vscales, block_table, seqlens, &o);
  if (rc) return rc;
  if ((rc = check_tensor(q, "q", ATTN_DTYPE_BF16, 3, false))) return rc;
  if ((rc = check_tensor(sinks, "sinks", ATTN_DTYPE_F32, 1, false))) return rc;
  if ((rc = check_tensor(out, "out", ATTN_DTYPE_BF16, 3, false))) return rc;
  const int64_t B = q->shape[0], Hq = q->shape[1];
  if (q->shape[2] != o.D) return fail(ATTN_EINVAL, "kpages head dim does not match q");
  for (int d = 0; d < 3; ++d)
    if (out->shape[d] != q->shape[d]) return fail(ATTN_EINVAL, "out shape does not match q");
  if (seqlens->shape[0] != B) return fail(ATTN_EINVAL, "block_table and seqlens must have B rows");
  if (sinks->shape[0] != Hq) return fail(ATTN_EINVAL, "sinks must have Hq entries");
  if (Hq > 1 && sinks->stride[0] != 1) return fail(ATTN_EINVAL, "sinks must be contiguous");
  if (Hq <= 0 || Hq % o.Hkv) return fail(ATTN_EINVAL, "Hq must be a positive multiple of Hkv");
  if (window < 1) return fail(ATTN_EINVAL, "window must be >= 1");
  if (!finite_pos(scale)) return fail(ATTN_EINVAL, "scale must be finite and > 0");
  if (Hq / o.Hkv > (o.D == 256 ? 8 : 16)) return fail(ATTN_EUNSUPPORTED, "Hq/Hkv too large for this head dim");
  if ((reinterpret_cast<uintptr_t>(q->data) % 4) || q->stride[0] % 2 || q->stride[1] % 2)
    return fail(ATTN_EINVAL, "q rows must be 4-byte aligned");
  if (B == 0) return ATTN_OK;
  PagedFp8Args a;
  a.q = static_cast<const __nv_bfloat16 *>(q->data);
  a.out = static_cast<__nv_bfloat16 *>(out->data);
  a.kpages = static_cast<const uint8_t *>(kpages->data);
  a.vpages = static_cast<const uint8_t *>(vpages->data);
  a.kscales = static_cast<const uint8_t *>(kscales->data);
  a.vscales = static_cast<const uint8_t *>(vscales->data);
  for (int d = 0; d < 2; ++d) {
    a.q_s[d] = q->stride[d];
    a.o_s[d] = out->stride[d];
    a.ks_s[d] = kscales->stride[d];
    a.vs_s[d] = vscales->stride[d];
  }
  for (int d = 0; d < 3; ++d) {
    a.kp_s[d] = kpages->stride[d];
    a.vp_s[d] = vpages->stride[d];
  }
  a.bt_s0 = block_table->stride[0];
  a.block_table = static_cast<const int *>(block_table->data);
  a.seqlens = static_cast<const int *>(seqlens->data);
  a.sinks = static_cast<const float *>(sinks->data);
  a.B = static_cast<int>(B);
  a.Hq = static_cast<int>(Hq);
  a.Hkv = static_cast<int>(o.Hkv);
  a.D = static_cast<int>(o.D);
  a.W = window;
  a.page = static_cast<int>(o.P);
  a.npages = static_cast<int>(o.NB);
  a.max_pages = static_cast<int>(o.MP);
  a.scale = scale;
  if ((rc = status_ptr(&a.status))) return rc;
  int sms;
  if ((rc = sm_count(&sms))) return rc;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const size_t bytes = paged_fp8_workspace_bytes(a, sms);
  if (bytes == 0) {
    const cudaError_t e = launch_decode_paged_fp8(a, nullptr, sms, st);
    return e == cudaSuccess ? ATTN_OK : fail_cuda(e, "attn_sink_decode_paged_fp8 launch");
  }
  cudaMemPool_t pool;
  if ((rc = workspace_pool(&pool))) return rc;
  void *ws = nullptr;
  if (take_injected_alloc_failure()) return fail(ATTN_ENOMEM, "decode workspace allocation failed (injected)");
  cudaError_t e = cudaMallocFromPoolAsync(&ws, bytes, pool, st);
  if (e != cudaSuccess) return fail_cuda(e, "decode workspace allocation");
  e = launch_decode_paged_fp8(a, ws, sms, st);
  const cudaError_t ef = cudaFreeAsync(ws, st);
  if (e != cudaSuccess) return fail_cuda(e, "attn_sink_decode_paged_fp8 launch");
  if (ef != cudaSuccess) return fail_cuda(ef, "decode workspace release");
  return ATTN_OK;
}

int attn_sink_fwd_extend(const attn_tensor *q, const attn_tensor *k, const attn_tensor *v,
                         const attn_tensor *cu_seqlens_q, const attn_tensor *cu_seqlens_k, int32_t max_seqlen_q,
                         const attn_tensor *sinks, int32_t window, float scale, attn_tensor *out, attn_tensor *lse,
                         void *stream) {
  clear_error();
  return extend_call(q, k, v, cu_seqlens_q, cu_seqlens_k, max_seqlen_q, sinks, window, scale, 0, out, lse, stream);
}

int attn_sink_fwd_extend_terms(const attn_tensor *q, const attn_tensor *k, const attn_tensor *v,
                               const attn_tensor *cu_seqlens_q, const attn_tensor *cu_seqlens_k,
                               int32_t max_seqlen_q, const attn_tensor *sinks, int32_t window, float scale,
                               int32_t terms, attn_tensor *out, attn_tensor *lse, void *stream) {
  clear_error();
  return extend_call(q, k, v, cu_seqlens_q, cu_seqlens_k, max_seqlen_q, sinks, window, scale, terms, out, lse, stream);
}

}  // extern "C"
