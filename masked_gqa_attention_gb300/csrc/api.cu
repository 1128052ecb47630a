// C ABI of the masked GQA attention library: argument validation and kernel
// dispatch. Allocates nothing and never synchronises; all work is enqueued on
// the caller's stream.
#include <cmath>
#include <cstdarg>
#include <cstdio>

#include "../../include/masked_gqa_attn.h"
#include "internal.h"

namespace mgqa {

static thread_local char g_detail[256] = "";

void clear_error_detail() { g_detail[0] = '\0'; }

mgqa_status fail(mgqa_status code, const char *fmt, ...) {
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(g_detail, sizeof(g_detail), fmt, ap);
  va_end(ap);
  return code;
}

int device_sm_count() {
  static std::atomic<int> cached[64];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 0;
  int n = cached[dev].load(std::memory_order_relaxed);
  if (n > 0) return n;
  if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n < 1) return 0;
  cached[dev].store(n, std::memory_order_relaxed);
  return n;
}

namespace {

bool aligned(const void *p, size_t n) { return (reinterpret_cast<uintptr_t>(p) % n) == 0; }

mgqa_status check_tensor(const char *name, const void *ptr, const int64_t *st, size_t esize) {
  if (!ptr) return fail(MGQA_ERR_INVALID_ARG, "%s is null", name);
  if (!aligned(ptr, 16)) return fail(MGQA_ERR_INVALID_ARG, "%s is not 16-byte aligned", name);
  for (int t = 0; t < 3; ++t) {
    if (st[t] < 0) return fail(MGQA_ERR_INVALID_ARG, "%s stride %d is negative", name, t);
    if ((st[t] * (int64_t)esize) % 16 != 0)
      return fail(MGQA_ERR_INVALID_ARG, "%s stride %d is not a multiple of 16 bytes", name, t);
  }
  return MGQA_OK;
}

mgqa_status validate(const mgqa_args *a, bool decode) {
  g_detail[0] = '\0';
  if (!a) return fail(MGQA_ERR_INVALID_ARG, "args is null");
  if (a->dtype != MGQA_BF16 && a->dtype != MGQA_FP32 && a->dtype != MGQA_FP16)
    return fail(MGQA_ERR_INVALID_ARG, "unknown dtype %d", (int)a->dtype);
  if (a->B < 1 || a->Hq < 1 || a->Hkv < 1 || a->Lq < 1 || a->Lk < 1)
    return fail(MGQA_ERR_INVALID_ARG, "B, Hq, Hkv, Lq, Lk must be >= 1");
  if (a->Hq % a->Hkv != 0) return fail(MGQA_ERR_INVALID_ARG, "Hq %% Hkv != 0");
  if (a->D != 64 && a->D != 128) return fail(MGQA_ERR_UNSUPPORTED, "head dim %d (64 or 128)", a->D);
  if (a->Lk > (1 << 24) || a->Lq > (1 << 24))
    return fail(MGQA_ERR_UNSUPPORTED, "sequence longer than 2^24");
  if ((int64_t)a->B * a->Hq * a->Lq > (int64_t)1 << 31)
    return fail(MGQA_ERR_UNSUPPORTED, "B*Hq*Lq too large");
  if (decode && a->Lq != 1) return fail(MGQA_ERR_INVALID_ARG, "decode needs Lq == 1");
  if (decode && a->Lk > kDecodeMaxLk)
    return fail(MGQA_ERR_UNSUPPORTED, "decode cache longer than %d slots", kDecodeMaxLk);
  if (!std::isfinite(a->scale)) return fail(MGQA_ERR_INVALID_ARG, "scale is not finite");
  const size_t es = a->dtype == MGQA_FP32 ? 4 : 2;
  mgqa_status st;
  if ((st = check_tensor("q", a->q, a->q_stride, es)) != MGQA_OK) return st;
  if ((st = check_tensor("k", a->k, a->k_stride, es)) != MGQA_OK) return st;
  if ((st = check_tensor("v", a->v, a->v_stride, es)) != MGQA_OK) return st;
  if ((st = check_tensor("out", a->out, a->o_stride, es)) != MGQA_OK) return st;
  if (a->mask_bits) {
    if (!aligned(a->mask_bits, 4)) return fail(MGQA_ERR_INVALID_ARG, "mask_bits misaligned");
    // a stride of 0 broadcasts one mask row over the queries (a key-padding
    // mask given as [B][1][W]) or one mask over the batch rows
    const int64_t W = (a->Lk + 31) / 32;
    if (a->mask_stride_b < 0 || a->mask_stride_q < 0)
      return fail(MGQA_ERR_INVALID_ARG, "negative mask stride");
    if (a->Lq > 1 && a->mask_stride_q != 0 && a->mask_stride_q < W)
      return fail(MGQA_ERR_INVALID_ARG, "mask_stride_q is neither 0 nor >= ceil(Lk/32)");
    if (a->B > 1 && a->mask_stride_b != 0 && a->mask_stride_b < W)
      return fail(MGQA_ERR_INVALID_ARG, "mask_stride_b is neither 0 nor >= ceil(Lk/32)");
  }
  if ((a->seg_q == nullptr) != (a->seg_k == nullptr))
    return fail(MGQA_ERR_INVALID_ARG, "seg_q and seg_k must be given together");
  if (a->seg_q && (!aligned(a->seg_q, 4) || !aligned(a->seg_k, 4)))
    return fail(MGQA_ERR_INVALID_ARG, "segment ids misaligned");
  if (a->kv_len && !aligned(a->kv_len, 4)) return fail(MGQA_ERR_INVALID_ARG, "kv_len misaligned");
  if (a->lse && !aligned(a->lse, 4)) return fail(MGQA_ERR_INVALID_ARG, "lse misaligned");
  if (a->dev_error && !aligned(a->dev_error, 4))
    return fail(MGQA_ERR_INVALID_ARG, "dev_error misaligned");
  return MGQA_OK;
}

// The fused rotary embedding of a call with head dim D, Hq / Hkv heads.
mgqa_status validate_rope(const mgqa_qk_rope *r, const mgqa_args &a, bool decode, FusedRope *out) {
  if (!r) return fail(MGQA_ERR_INVALID_ARG, "rope is null");
  if (!r->inv_freq || !aligned(r->inv_freq, 4))
    return fail(MGQA_ERR_INVALID_ARG, "rope: inv_freq missing or misaligned");
  if (r->rot_dim < 2 || r->rot_dim > a.D || (r->rot_dim & 1))
    return fail(MGQA_ERR_INVALID_ARG, "rope: rot_dim must be even and in [2, D]");
  if (r->q_heads < 1 || r->q_heads > a.Hq)
    return fail(MGQA_ERR_INVALID_ARG, "rope: q_heads must be in [1, Hq]");
  if (decode && (r->k_heads < 0 || r->k_heads > a.Hkv))
    return fail(MGQA_ERR_INVALID_ARG, "rope: k_heads must be in [0, Hkv]");
  if (r->positions && !aligned(r->positions, 4))
    return fail(MGQA_ERR_INVALID_ARG, "rope: positions misaligned");
  if ((r->q_norm_weight && !aligned(r->q_norm_weight, 4)) ||
      (r->k_norm_weight && !aligned(r->k_norm_weight, 4)))
    return fail(MGQA_ERR_INVALID_ARG, "rope: norm weight misaligned");
  if ((r->q_norm_weight || r->k_norm_weight) && !(std::isfinite(r->norm_eps) && r->norm_eps >= 0.f))
    return fail(MGQA_ERR_INVALID_ARG, "rope: norm_eps must be finite and >= 0");
  out->inv_freq = r->inv_freq;
  out->positions = r->positions;
  out->half = r->rot_dim / 2;
  out->interleaved = r->interleaved != 0;
  out->q_heads = r->q_heads;
  out->k_heads = decode ? r->k_heads : 0;
  out->q_norm = r->q_norm_weight;
  out->k_norm = decode ? r->k_norm_weight : nullptr;
  out->eps = r->norm_eps;
  return MGQA_OK;
}

mgqa_status validate_append(const mgqa_args *args, const void *k_new, const void *v_new,
                            const int64_t *k_new_stride, const int64_t *v_new_stride,
                            int32_t *kv_len_out) {
  mgqa_status st = validate(args, true);
  if (st != MGQA_OK) return st;
  if (!args->kv_len) return fail(MGQA_ERR_INVALID_ARG, "append needs kv_len");
  if (args->mask_bits || args->seg_q)
    return fail(MGQA_ERR_INVALID_ARG, "append takes the kv_len form only");
  if (!k_new || !v_new || !k_new_stride || !v_new_stride)
    return fail(MGQA_ERR_INVALID_ARG, "append needs k_new, v_new and their strides");
  const size_t es = args->dtype == MGQA_FP32 ? 4 : 2;
  if ((reinterpret_cast<uintptr_t>(k_new) % 16) || (reinterpret_cast<uintptr_t>(v_new) % 16))
    return fail(MGQA_ERR_INVALID_ARG, "k_new / v_new not 16-byte aligned");
  for (int t = 0; t < 2; ++t)
    if (k_new_stride[t] < 0 || v_new_stride[t] < 0 || (k_new_stride[t] * (int64_t)es) % 16 ||
        (v_new_stride[t] * (int64_t)es) % 16)
      return fail(MGQA_ERR_INVALID_ARG, "k_new / v_new strides must be multiples of 16 bytes");
  if (kv_len_out && kv_len_out == args->kv_len)
    return fail(MGQA_ERR_INVALID_ARG, "kv_len_out must not alias kv_len");
  if (kv_len_out && (reinterpret_cast<uintptr_t>(kv_len_out) % 4))
    return fail(MGQA_ERR_INVALID_ARG, "kv_len_out misaligned");
  return MGQA_OK;
}

mgqa_status check_window(int32_t window, int32_t sinks, int32_t least) {
  if (window < least) return fail(MGQA_ERR_INVALID_ARG, "window must be >= %d", least);
  if (sinks < 0) return fail(MGQA_ERR_INVALID_ARG, "sinks must be >= 0");
  return MGQA_OK;
}

// One token or a tree over a cache: args and pages.
mgqa_status validate_cached(const mgqa_args *args, const mgqa_pages *pages) {
  mgqa_status st = validate(args, false);
  if (st != MGQA_OK) return st;
  if (!args->kv_len) return fail(MGQA_ERR_INVALID_ARG, "kv_len is required");
  if (args->mask_bits || args->seg_q || args->causal)
    return fail(MGQA_ERR_INVALID_ARG, "the cache forms take no mask_bits, segment ids or causal");
  if (pages) {
    if (!pages->table || !aligned(pages->table, 4))
      return fail(MGQA_ERR_INVALID_ARG, "page table missing or misaligned");
    if (pages->num_pages < 1 || pages->page_size < 1 || pages->max_pages < 1)
      return fail(MGQA_ERR_INVALID_ARG, "num_pages, page_size and max_pages must be >= 1");
    if ((int64_t)pages->page_size * pages->max_pages != args->Lk)
      return fail(MGQA_ERR_INVALID_ARG, "Lk is not max_pages * page_size");
    if (args->B > 1 && pages->table_stride < pages->max_pages)
      return fail(MGQA_ERR_INVALID_ARG, "table_stride < max_pages");
  }
  return MGQA_OK;
}

mgqa_status check_new_rows(const void *k, const void *v, const int64_t *ks, const int64_t *vs, int dims, size_t es) {
  if (!k || !v || !aligned(k, 16) || !aligned(v, 16))
    return fail(MGQA_ERR_INVALID_ARG, "k_new / v_new missing or not 16-byte aligned");
  if (!ks || !vs) return fail(MGQA_ERR_INVALID_ARG, "k_new / v_new strides missing");
  for (int t = 0; t < dims; ++t)
    if (ks[t] < 0 || vs[t] < 0 || (ks[t] * (int64_t)es) % 16 || (vs[t] * (int64_t)es) % 16)
      return fail(MGQA_ERR_INVALID_ARG, "k_new / v_new strides must be non-negative multiples of 16 bytes");
  return MGQA_OK;
}

mgqa_status validate_tree(const mgqa_args *a, const mgqa_tree *tree) {
  if (!tree) return fail(MGQA_ERR_INVALID_ARG, "tree is null");
  if (a->Lq > kMaxDraftsHost)
    return fail(MGQA_ERR_UNSUPPORTED, "%d drafted tokens (at most %d)", a->Lq, kMaxDraftsHost);
  const mgqa_status st = check_new_rows(tree->k_new, tree->v_new, tree->k_stride, tree->v_stride, 3,
                                        a->dtype == MGQA_FP32 ? 4 : 2);
  if (st != MGQA_OK) return st;
  if (tree->bits) {
    const int64_t W = (a->Lq + 31) / 32;
    if (!aligned(tree->bits, 4)) return fail(MGQA_ERR_INVALID_ARG, "tree bits misaligned");
    if ((a->B > 1 && tree->bits_stride_b != 0 && tree->bits_stride_b < W) || tree->bits_stride_b < 0 ||
        (a->Lq > 1 && tree->bits_stride_t != 0 && tree->bits_stride_t < W) || tree->bits_stride_t < 0)
      return fail(MGQA_ERR_INVALID_ARG, "tree bits: a stride is neither 0 nor >= ceil(Lq/32)");
  }
  if (tree->len && !aligned(tree->len, 4)) return fail(MGQA_ERR_INVALID_ARG, "tree len misaligned");
  return MGQA_OK;
}

// Do n ints at a and m ints at b share any? (a null b shares none)
bool ints_overlap(const int32_t *a, int64_t n, const int32_t *b, int64_t m) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return b && x < y + 4 * (uintptr_t)m && y < x + 4 * (uintptr_t)n;
}

mgqa_status check_workspace(const void *ws, size_t have, size_t need) {
  if (!ws || !aligned(ws, 16)) return fail(MGQA_ERR_INVALID_ARG, "workspace missing or not 16-byte aligned");
  if (have < need) return fail(MGQA_ERR_INVALID_ARG, "workspace of %zu bytes, %zu needed", have, need);
  return MGQA_OK;
}

// A cache description; `counted`: page table and reference counts are needed.
mgqa_status validate_cache(const mgqa_cache *c, bool counted) {
  g_detail[0] = '\0';
  if (!c) return fail(MGQA_ERR_INVALID_ARG, "cache is null");
  if (c->dtype != MGQA_BF16 && c->dtype != MGQA_FP32 && c->dtype != MGQA_FP16)
    return fail(MGQA_ERR_INVALID_ARG, "unknown dtype %d", (int)c->dtype);
  if (c->layers < 1 || c->num_pages < 1 || c->Hkv < 1 || c->page_size < 1 || c->D < 1 || c->rows < 1)
    return fail(MGQA_ERR_INVALID_ARG, "layers, num_pages, Hkv, page_size, D and rows must be >= 1");
  const size_t es = c->dtype == MGQA_FP32 ? 4 : 2;
  if ((c->D * es) % 16) return fail(MGQA_ERR_UNSUPPORTED, "a row of D elements is not a multiple of 16 bytes");
  if (!c->k || !c->v || !aligned(c->k, 16) || !aligned(c->v, 16))
    return fail(MGQA_ERR_INVALID_ARG, "cache k / v missing or not 16-byte aligned");
  for (int t = 0; t < 4; ++t)
    if (c->k_stride[t] < 0 || c->v_stride[t] < 0 || (c->k_stride[t] * (int64_t)es) % 16 ||
        (c->v_stride[t] * (int64_t)es) % 16)
      return fail(MGQA_ERR_INVALID_ARG, "cache strides must be non-negative multiples of 16 bytes");
  if (c->kv_len && !aligned(c->kv_len, 4)) return fail(MGQA_ERR_INVALID_ARG, "kv_len misaligned");
  if (c->dev_error && !aligned(c->dev_error, 4)) return fail(MGQA_ERR_INVALID_ARG, "dev_error misaligned");
  if (c->page_table) {
    if (!aligned(c->page_table, 4)) return fail(MGQA_ERR_INVALID_ARG, "page table misaligned");
    if (c->max_pages < 1) return fail(MGQA_ERR_INVALID_ARG, "max_pages must be >= 1");
    if (c->rows > 1 && c->table_stride < c->max_pages)
      return fail(MGQA_ERR_INVALID_ARG, "table_stride < max_pages");
    if ((int64_t)c->max_pages * c->page_size > (1 << 24))
      return fail(MGQA_ERR_UNSUPPORTED, "a request of more than 2^24 slots");
  } else {
    if (counted) return fail(MGQA_ERR_INVALID_ARG, "a page table is required");
    if (c->num_pages != c->rows) return fail(MGQA_ERR_INVALID_ARG, "static cache: num_pages is not rows");
    if (c->page_size > (1 << 24)) return fail(MGQA_ERR_UNSUPPORTED, "a request of more than 2^24 slots");
  }
  if (counted) {
    if (!c->ref || !aligned(c->ref, 4)) return fail(MGQA_ERR_INVALID_ARG, "ref missing or misaligned");
    if (c->num_pages > kMaxPages) return fail(MGQA_ERR_UNSUPPORTED, "more than %d pages", kMaxPages);
    if ((int64_t)c->page_size * (int64_t)(c->D * es / 16) > kMaxPagePieces)
      return fail(MGQA_ERR_UNSUPPORTED, "a page of more than 2^34 bytes of a head");
  }
  return MGQA_OK;
}

// A cache of records in 4 bits: dtype and D are those of the rows that are appended,
// the strides bytes.
mgqa_status validate_cache_q4(const mgqa_cache *c) {
  g_detail[0] = '\0';
  if (!c) return fail(MGQA_ERR_INVALID_ARG, "cache is null");
  if (c->D != 64 && c->D != 128) return fail(MGQA_ERR_UNSUPPORTED, "head dim %d (64 or 128)", c->D);
  for (int t = 0; t < 4; ++t)
    if (c->k_stride[t] % 16 || c->v_stride[t] % 16)
      return fail(MGQA_ERR_INVALID_ARG, "cache strides must be non-negative multiples of 16 bytes");
  return validate_cache(c, false);
}

// The last Lq cached tokens over a cache (of records, or of the call's type).
mgqa_status validate_last(const mgqa_args *args, const mgqa_pages *pages, int32_t window, int32_t sinks, bool q4,
                          bool values) {
  g_detail[0] = '\0';
  if (!args) return fail(MGQA_ERR_INVALID_ARG, "args is null");
  mgqa_args a = *args;
  if (!values) {  // the call has no values and no output
    a.v = a.k;
    a.out = const_cast<void *>(a.q);
    for (int t = 0; t < 3; ++t) {
      a.v_stride[t] = a.k_stride[t];
      a.o_stride[t] = a.q_stride[t];
    }
  }
  if (q4)
    for (int t = 0; t < 3; ++t)
      if (a.k_stride[t] % 16 || a.v_stride[t] % 16)
        return fail(MGQA_ERR_INVALID_ARG, "strides of records must be non-negative multiples of 16 bytes");
  mgqa_status st = validate_cached(&a, pages);
  if (st != MGQA_OK) return st;
  if (a.Lq > kMaxDraftsHost) return fail(MGQA_ERR_UNSUPPORTED, "%d queries a request (at most %d)", a.Lq, kMaxDraftsHost);
  return check_window(window, sinks, 0);
}

// fp32 [n0][n1][n2][slots] with strides st.
mgqa_status check_weight(const char *name, const float *w, const int64_t *st, const int64_t *n, int64_t slots) {
  if (!w || !st || !aligned(w, 4)) return fail(MGQA_ERR_INVALID_ARG, "%s or its strides missing or misaligned", name);
  if (slots < 1) return fail(MGQA_ERR_INVALID_ARG, "weight_slots must be >= 1");
  // the heads' rows may not overlap: in some order of the dimensions, each stride is
  // at least what the smaller ones span
  int64_t span = slots;
  bool done[3] = {n[0] == 1, n[1] == 1, n[2] == 1};
  for (int k = 0; k < 3; ++k) {
    int next = -1;
    for (int t = 0; t < 3; ++t)
      if (!done[t] && (next < 0 || st[t] < st[next])) next = t;
    if (next < 0) break;
    if (st[next] < span || st[next] > ((int64_t)1 << 60) / n[next])
      return fail(MGQA_ERR_INVALID_ARG, "%s: the slots of two heads overlap", name);
    span += (n[next] - 1) * st[next];
    done[next] = true;
  }
  return MGQA_OK;
}

mgqa_status validate_evict(const mgqa_cache *c, int32_t budget, int32_t sinks, int32_t recent) {
  mgqa_status st = validate_cache(c, false);
  if (st != MGQA_OK) return st;
  if (c->ref && !aligned(c->ref, 4)) return fail(MGQA_ERR_INVALID_ARG, "ref misaligned");
  if (c->ref && !c->page_table) return fail(MGQA_ERR_INVALID_ARG, "ref without a page table");
  if (budget < 1 || budget > (1 << 24)) return fail(MGQA_ERR_INVALID_ARG, "budget must be in [1, 2^24]");
  if (sinks < 0 || recent < 0 || (int64_t)sinks + recent > budget)
    return fail(MGQA_ERR_INVALID_ARG, "sinks and recent must be >= 0 and sum to at most the budget");
  if ((int64_t)c->layers * c->rows * c->Hkv > (1 << 26))
    return fail(MGQA_ERR_UNSUPPORTED, "layers x requests x KV heads past 2^26");
  return MGQA_OK;
}

}  // namespace
}  // namespace mgqa

extern "C" {

mgqa_status masked_gqa_attn_prefill(const mgqa_args *args, cudaStream_t stream) {
  mgqa_status st = mgqa::validate(args, false);
  if (st != MGQA_OK) return st;
  if (args->dtype != MGQA_FP32) return mgqa::launch_prefill_tc(*args, stream);
  return mgqa::launch_prefill_simt(*args, stream);
}

size_t masked_gqa_attn_decode_workspace_size(const mgqa_args *args) {
  if (mgqa::validate(args, true) != MGQA_OK) return 0;
  return mgqa::kDecodeWorkspaceBytes;
}

mgqa_status masked_gqa_attn_decode(const mgqa_args *args, void *workspace, size_t workspace_bytes,
                                   cudaStream_t stream) {
  (void)workspace;  // merged on chip: nothing is read or written there
  (void)workspace_bytes;
  mgqa_status st = mgqa::validate(args, true);
  if (st != MGQA_OK) return st;
  return mgqa::launch_decode(*args, stream);
}

mgqa_status masked_gqa_attn_decode_append(const mgqa_args *args, const void *k_new,
                                          const void *v_new, const int64_t *k_new_stride,
                                          const int64_t *v_new_stride, int32_t *kv_len_out,
                                          void *workspace, size_t workspace_bytes,
                                          cudaStream_t stream) {
  (void)workspace;
  (void)workspace_bytes;
  const mgqa_status st = mgqa::validate_append(args, k_new, v_new, k_new_stride, v_new_stride,
                                               kv_len_out);
  if (st != MGQA_OK) return st;
  return mgqa::launch_decode_append(*args, k_new, v_new, k_new_stride, v_new_stride, kv_len_out,
                                    stream);
}

mgqa_status masked_gqa_attn_decode_append_rope(const mgqa_args *args, const void *k_new,
                                               const void *v_new, const int64_t *k_new_stride,
                                               const int64_t *v_new_stride, int32_t *kv_len_out,
                                               const mgqa_qk_rope *rope, void *workspace,
                                               size_t workspace_bytes, cudaStream_t stream) {
  (void)workspace;
  (void)workspace_bytes;
  mgqa_status st = mgqa::validate_append(args, k_new, v_new, k_new_stride, v_new_stride,
                                         kv_len_out);
  if (st != MGQA_OK) return st;
  mgqa::FusedRope fr;
  if ((st = mgqa::validate_rope(rope, *args, true, &fr)) != MGQA_OK) return st;
  return mgqa::launch_decode_append(*args, k_new, v_new, k_new_stride, v_new_stride, kv_len_out,
                                    stream, fr);
}

mgqa_status masked_gqa_attn_prefill_rope(const mgqa_args *args, const mgqa_qk_rope *rope,
                                         cudaStream_t stream) {
  mgqa_status st = mgqa::validate(args, false);
  if (st != MGQA_OK) return st;
  if (args->dtype == MGQA_FP32)
    return mgqa::fail(MGQA_ERR_UNSUPPORTED,
                      "the fused rotary embedding runs on the bf16 / fp16 path; rotate fp32 inputs "
                      "with masked_gqa_rope");
  mgqa::FusedRope fr;
  if ((st = mgqa::validate_rope(rope, *args, false, &fr)) != MGQA_OK) return st;
  // the kernel keeps a query row in registers, which needs the pairing fixed
  // at compile time: half-split rotations over D, D/2 or D/4 features
  if (!fr.interleaved && fr.half != args->D / 2 && fr.half != args->D / 4 && fr.half != args->D / 8)
    return mgqa::fail(MGQA_ERR_UNSUPPORTED,
                      "fused prefill: half-split rotary dims must be D, D/2 or D/4 (rotate with "
                      "masked_gqa_rope for other widths)");
  return mgqa::launch_prefill_tc(*args, stream, fr);
}

mgqa_status masked_gqa_attn_prefill_window(const mgqa_args *args, int32_t window, int32_t sinks,
                                           cudaStream_t stream) {
  mgqa_status st = mgqa::validate(args, false);
  if (st != MGQA_OK) return st;
  if ((st = mgqa::check_window(window, sinks, 1)) != MGQA_OK) return st;
  // the tiles come by TMA, which knows no stride of 0 (fp32 reads q without it)
  if (!mgqa::plain_strides(args->k_stride, args->B, args->Hkv, args->Lk) ||
      !mgqa::plain_strides(args->v_stride, args->B, args->Hkv, args->Lk) ||
      (args->dtype != MGQA_FP32 && !mgqa::plain_strides(args->q_stride, args->B, args->Hq, args->Lq)))
    return mgqa::fail(MGQA_ERR_UNSUPPORTED, "windowed prefill: a tensor expanded over a dimension");
  const mgqa::WindowRule win{window < mgqa::kWidestWindow ? window : mgqa::kWidestWindow,
                             sinks < args->Lk ? sinks : args->Lk};
  if (args->dtype != MGQA_FP32) return mgqa::launch_prefill_tc(*args, stream, mgqa::FusedRope(), win);
  return mgqa::launch_prefill_window_f32(*args, win, stream);
}

size_t masked_gqa_attn_cache_workspace_size(void) { return mgqa::cache_attn_workspace_bytes(); }

mgqa_status masked_gqa_attn_decode_window(const mgqa_args *args, const mgqa_pages *pages, int32_t window,
                                          int32_t sinks, void *workspace, size_t workspace_bytes,
                                          cudaStream_t stream) {
  mgqa_status st = mgqa::validate_cached(args, pages);
  if (st != MGQA_OK) return st;
  if (args->Lq != 1) return mgqa::fail(MGQA_ERR_INVALID_ARG, "decode needs Lq == 1");
  if ((st = mgqa::check_window(window, sinks, 1)) != MGQA_OK) return st;
  if ((st = mgqa::check_workspace(workspace, workspace_bytes, mgqa::cache_attn_workspace_bytes())) != MGQA_OK)
    return st;
  return mgqa::launch_cache_attn(*args, pages, nullptr, window, sinks, workspace, stream);
}

mgqa_status masked_gqa_attn_decode_tree(const mgqa_args *args, const mgqa_pages *pages, const mgqa_tree *tree,
                                        int32_t window, int32_t sinks, void *workspace, size_t workspace_bytes,
                                        cudaStream_t stream) {
  mgqa_status st = mgqa::validate_cached(args, pages);
  if (st != MGQA_OK) return st;
  if ((st = mgqa::validate_tree(args, tree)) != MGQA_OK) return st;
  if ((st = mgqa::check_window(window, sinks, 0)) != MGQA_OK) return st;
  if ((st = mgqa::check_workspace(workspace, workspace_bytes, mgqa::cache_attn_workspace_bytes())) != MGQA_OK)
    return st;
  return mgqa::launch_cache_attn(*args, pages, tree, window, sinks, workspace, stream);
}

namespace {

mgqa_status append_rows(const mgqa_cache *cache, const void *k_new, const void *v_new, const int64_t *k_new_stride,
                        const int64_t *v_new_stride, int32_t T, const int32_t *index, const int32_t *count,
                        int32_t *kv_len_out, bool q4, cudaStream_t stream) {
  mgqa_status st = q4 ? mgqa::validate_cache_q4(cache) : mgqa::validate_cache(cache, false);
  if (st != MGQA_OK) return st;
  if (!cache->kv_len || !kv_len_out) return mgqa::fail(MGQA_ERR_INVALID_ARG, "kv_len and kv_len_out are required");
  if (!mgqa::aligned(kv_len_out, 4) || !mgqa::aligned(index, 4) || !mgqa::aligned(count, 4))
    return mgqa::fail(MGQA_ERR_INVALID_ARG, "kv_len_out, index or count misaligned");
  if (T < 1 || T > (1 << 24)) return mgqa::fail(MGQA_ERR_INVALID_ARG, "T must be in [1, 2^24]");
  // one block writes a request's new length while others still read the inputs
  const int64_t rows = cache->rows, entries = (rows - 1) * cache->table_stride + cache->max_pages;
  if (mgqa::ints_overlap(kv_len_out, rows, cache->kv_len, rows) ||
      mgqa::ints_overlap(kv_len_out, rows, count, rows) || mgqa::ints_overlap(kv_len_out, rows, index, rows * T) ||
      mgqa::ints_overlap(kv_len_out, rows, cache->page_table, entries))
    return mgqa::fail(MGQA_ERR_INVALID_ARG, "kv_len_out must not overlap kv_len, count, index or the page table");
  if ((st = mgqa::check_new_rows(k_new, v_new, k_new_stride, v_new_stride, 4, cache->dtype == MGQA_FP32 ? 4 : 2)) !=
      MGQA_OK)
    return st;
  return mgqa::launch_cache_append(*cache, k_new, v_new, k_new_stride, v_new_stride, T, index, count, kv_len_out, q4,
                                   stream);
}

}  // namespace

mgqa_status masked_gqa_cache_append(const mgqa_cache *cache, const void *k_new, const void *v_new,
                                    const int64_t *k_new_stride, const int64_t *v_new_stride, int32_t T,
                                    const int32_t *index, const int32_t *count, int32_t *kv_len_out,
                                    cudaStream_t stream) {
  return append_rows(cache, k_new, v_new, k_new_stride, v_new_stride, T, index, count, kv_len_out, false, stream);
}

mgqa_status masked_gqa_cache_append_q4(const mgqa_cache *cache, const void *k_new, const void *v_new,
                                       const int64_t *k_new_stride, const int64_t *v_new_stride, int32_t T,
                                       const int32_t *index, const int32_t *count, int32_t *kv_len_out,
                                       cudaStream_t stream) {
  return append_rows(cache, k_new, v_new, k_new_stride, v_new_stride, T, index, count, kv_len_out, true, stream);
}

mgqa_status masked_gqa_attn_decode_q4(const mgqa_args *args, const mgqa_pages *pages, int32_t window, int32_t sinks,
                                      void *workspace, size_t workspace_bytes, cudaStream_t stream) {
  mgqa_status st = mgqa::validate_last(args, pages, window, sinks, true, true);
  if (st != MGQA_OK) return st;
  if ((st = mgqa::check_workspace(workspace, workspace_bytes, mgqa::cache_attn_workspace_bytes())) != MGQA_OK)
    return st;
  return mgqa::launch_attn_q4(*args, pages, window, sinks, workspace, stream);
}

mgqa_status masked_gqa_attn_cache_weights(const mgqa_args *args, const mgqa_pages *pages, int32_t window,
                                          int32_t sinks, int32_t q4, float *weight, const int64_t *weight_stride,
                                          int32_t weight_slots, cudaStream_t stream) {
  mgqa_status st = mgqa::validate_last(args, pages, window, sinks, q4 != 0, false);
  if (st != MGQA_OK) return st;
  if (!args->lse) return mgqa::fail(MGQA_ERR_INVALID_ARG, "lse is required");
  const int64_t heads[3] = {1, args->B, args->Hkv}, strides[3] = {0, weight_stride ? weight_stride[0] : 0,
                                                                  weight_stride ? weight_stride[1] : 0};
  if ((st = mgqa::check_weight("weight", weight, weight_stride ? strides : nullptr, heads, weight_slots)) != MGQA_OK)
    return st;
  return mgqa::launch_cache_weights(*args, pages, window, sinks, q4 != 0, weight, weight_stride, weight_slots, stream);
}

size_t masked_gqa_cache_evict_workspace_size(const mgqa_cache *cache, int32_t budget) {
  if (mgqa::validate_evict(cache, budget, 0, 0) != MGQA_OK) return 0;
  return mgqa::cache_evict_workspace_bytes(*cache, budget);
}

mgqa_status masked_gqa_cache_evict(const mgqa_cache *cache, const float *weight, const int64_t *weight_stride,
                                   float *weight_out, const int64_t *weight_out_stride, int32_t weight_slots,
                                   int32_t budget, int32_t sinks, int32_t recent, int32_t *kv_len_out, void *workspace,
                                   size_t workspace_bytes, cudaStream_t stream) {
  mgqa_status st = mgqa::validate_evict(cache, budget, sinks, recent);
  if (st != MGQA_OK) return st;
  if (!cache->kv_len || !kv_len_out || !mgqa::aligned(kv_len_out, 4))
    return mgqa::fail(MGQA_ERR_INVALID_ARG, "kv_len or kv_len_out missing or misaligned");
  const int64_t rows = cache->rows, n[3] = {cache->layers, rows, cache->Hkv};
  const int64_t slots = weight_slots;
  if ((st = mgqa::check_weight("weight", weight, weight_stride, n, slots)) != MGQA_OK) return st;
  if ((st = mgqa::check_weight("weight_out", weight_out, weight_out_stride, n, slots)) != MGQA_OK) return st;
  const auto span = [&](const int64_t *t) { return (n[0] - 1) * t[0] + (n[1] - 1) * t[1] + (n[2] - 1) * t[2] + slots; };
  const auto as_ints = [](const void *p) { return static_cast<const int32_t *>(p); };
  bool same = weight == weight_out;
  for (int t = 0; t < 3; ++t) same = same && (n[t] == 1 || weight_stride[t] == weight_out_stride[t]);
  if (!same && mgqa::ints_overlap(as_ints(weight), span(weight_stride), as_ints(weight_out), span(weight_out_stride)))
    return mgqa::fail(MGQA_ERR_INVALID_ARG, "weight_out must be weight itself or not overlap it");
  if (cache->kv_len != kv_len_out && mgqa::ints_overlap(cache->kv_len, rows, kv_len_out, rows))
    return mgqa::fail(MGQA_ERR_INVALID_ARG, "kv_len_out must be kv_len itself or not overlap it");
  if (mgqa::ints_overlap(kv_len_out, rows, as_ints(weight_out), span(weight_out_stride)) ||
      mgqa::ints_overlap(kv_len_out, rows, cache->page_table, (rows - 1) * cache->table_stride + cache->max_pages))
    return mgqa::fail(MGQA_ERR_INVALID_ARG, "kv_len_out must not overlap the weights or the page table");
  if ((st = mgqa::check_workspace(workspace, workspace_bytes, mgqa::cache_evict_workspace_bytes(*cache, budget))) !=
      MGQA_OK)
    return st;
  return mgqa::launch_cache_evict(*cache, weight, weight_stride, weight_out, weight_out_stride, weight_slots, budget,
                                  sinks, recent, kv_len_out, workspace, stream);
}

size_t masked_gqa_cache_workspace_size(const mgqa_cache *cache, int32_t n) {
  if (mgqa::validate_cache(cache, true) != MGQA_OK) return 0;
  if (n < 0 || n > mgqa::kMaxForks) {
    mgqa::fail(MGQA_ERR_INVALID_ARG, "n must be in [0, %d]", mgqa::kMaxForks);
    return 0;
  }
  return mgqa::cache_pages_workspace_bytes(*cache, n);
}

mgqa_status masked_gqa_cache_fork(const mgqa_cache *cache, int32_t n, const int32_t *src, const int32_t *dst,
                                  int32_t extra, void *workspace, size_t workspace_bytes, cudaStream_t stream) {
  mgqa_status st = mgqa::validate_cache(cache, true);
  if (st != MGQA_OK) return st;
  if (!cache->kv_len) return mgqa::fail(MGQA_ERR_INVALID_ARG, "kv_len is required");
  if (n < 0 || n > mgqa::kMaxForks) return mgqa::fail(MGQA_ERR_INVALID_ARG, "n must be in [0, %d]", mgqa::kMaxForks);
  if (extra < 0 || extra > (1 << 24)) return mgqa::fail(MGQA_ERR_INVALID_ARG, "extra must be in [0, 2^24]");
  if (n == 0) return MGQA_OK;
  if (!src || !dst || !mgqa::aligned(src, 4) || !mgqa::aligned(dst, 4))
    return mgqa::fail(MGQA_ERR_INVALID_ARG, "src or dst missing or misaligned");
  if ((st = mgqa::check_workspace(workspace, workspace_bytes, mgqa::cache_pages_workspace_bytes(*cache, n))) !=
      MGQA_OK)
    return st;
  return mgqa::launch_cache_fork(*cache, n, src, dst, extra, workspace, stream);
}

mgqa_status masked_gqa_cache_compact(const mgqa_cache *cache, int32_t *page_table_out, int64_t table_out_stride,
                                     int32_t *ref_out, int32_t *used_out, void *workspace, size_t workspace_bytes,
                                     cudaStream_t stream) {
  mgqa_status st = mgqa::validate_cache(cache, true);
  if (st != MGQA_OK) return st;
  if (!page_table_out || !ref_out || !mgqa::aligned(page_table_out, 4) || !mgqa::aligned(ref_out, 4) ||
      !mgqa::aligned(used_out, 4))
    return mgqa::fail(MGQA_ERR_INVALID_ARG, "page_table_out or ref_out missing or misaligned");
  if (cache->rows > 1 && table_out_stride < cache->max_pages)
    return mgqa::fail(MGQA_ERR_INVALID_ARG, "table_out_stride < max_pages");
  if (page_table_out == cache->page_table && cache->rows > 1 && table_out_stride != cache->table_stride)
    return mgqa::fail(MGQA_ERR_INVALID_ARG, "an aliased page_table_out needs page_table's stride");
  if ((st = mgqa::check_workspace(workspace, workspace_bytes, mgqa::cache_pages_workspace_bytes(*cache, 0))) !=
      MGQA_OK)
    return st;
  return mgqa::launch_cache_compact(*cache, page_table_out, table_out_stride, ref_out, used_out, workspace, stream);
}

const char *mgqa_status_string(mgqa_status s) {
  switch (s) {
    case MGQA_OK: return "ok";
    case MGQA_ERR_INVALID_ARG: return "invalid argument";
    case MGQA_ERR_UNSUPPORTED: return "unsupported";
    case MGQA_ERR_CUDA: return "CUDA error";
    case MGQA_ERR_TIMEOUT: return "device wait timed out";
    case MGQA_ERR_DEVICE_CHECK: return "device bounds check failed (debug library)";
  }
  return "unknown status";
}

const char *mgqa_last_error_detail(void) { return mgqa::g_detail; }

int32_t mgqa_abi_version(void) { return MGQA_ABI_VERSION; }

}  // extern "C"
