// Attention of one new token (sliding window and sinks), or of a tree of
// drafted tokens, per request over a key/value cache in slots or pages.
//
// Per request b with n = kv_len[b] cached tokens, KV head g and query row
// (draft t, query head h of g), at position p_t = n + depth(t) (one token:
// n - 1, the last cached one):
//   s_j = scale <q, k_j>   over cached j < n with p_t - j < window or j < sinks
//                          and over the drafts t sees (the same rule on p)
//   out = sum_j softmax(s)_j v_j,   lse = log sum_j exp(s_j)
// One pass over the keys with a running maximum and sum per row; a run of
// tiles that ends inside a unit leaves (m, l, O) and the merge kernel joins
// them (cache_sched.cuh has the split).
//
// What bounds it: every visible key and value row is read once per KV head,
// 4 R D operations per key for its R = T * Hq / Hkv query rows, so up to about
// R = 64 the reads are the floor, and beyond a few hundred the products. Three
// kernels, by the type and R (launch_cache_attn): cache_attn_tma.cu (mma.sync),
// cache_attn_tc.cu (tensor memory), cache_attn_f32.cu (CUDA cores); all over
// slots or pages of any size. This file picks one and has the kernel that joins
// the partial results.
#include <algorithm>
#include <cmath>

#include "cache_sched.cuh"

namespace mgqa {
namespace {

// ---- joining the partial results -------------------------------------------------

constexpr int kMergeThreads = 128;

// Block (unit or run, 16 rows, 32 features): joins the pieces of the unit, if it
// was cut, in the order of the runs. A thread has four features of a row; partial
// results are read in runs of 16 rows x 16 bytes.
template <typename T, int D, int BR>
__global__ void __launch_bounds__(kMergeThreads)
cache_merge_kernel(const __grid_constant__ CacheAttnParams p) {
  const int r = blockIdx.y * 16 + threadIdx.x % 16, d = (blockIdx.z * 8 + threadIdx.x / 16) * 4;
  grid_dependency_wait();
  allow_dependents();
  const int4 cut = __ldcg(p.cuts + blockIdx.x);
  if (cut.z < 0) return;
  const int b = cut.x, unit = cut.y, last = cut.z, first = cut.w, units = p.Hkv * p.RB;
  // (an attention kernel whose waits gave up may have left no word: nothing is joined then)
  if ((unsigned)b >= (unsigned)p.B || (unsigned)unit >= (unsigned)units || (unsigned)first >= (unsigned)p.grid ||
      last >= p.grid || (p.by_unit ? b * units + unit : first) != (int)blockIdx.x)
    return;
  const int row0 = (unit % p.RB) * p.block_rows, rows = min(p.block_rows, p.R - row0);
  if (r >= rows) return;
  const PieceOut po{true, 0, b, unit / p.RB, row0, rows};
  const float2 *ml = p.part_ml + r;
  const float *po_ = p.part_o + (d / 4) * (BR * 4) + r * 4;
  float m = -INFINITY, l = 0.f;
  float acc[4] = {0.f, 0.f, 0.f, 0.f};
  constexpr int U = 8;  // partial results in flight
  for (int x = first; x <= last; x += U) {
    float2 a[U];
    float4 v[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      a[u] = make_float2(-INFINITY, 0.f);
      v[u] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (x + u <= last) {
        const int64_t slot = 2 * (x + u) + (x + u == first);
        a[u] = ml[slot * BR];
        v[u] = *reinterpret_cast<const float4 *>(po_ + slot * (BR * D));
      }
    }
    float mn = m;
#pragma unroll
    for (int u = 0; u < U; ++u) mn = fmaxf(mn, a[u].x);
    if (mn == -INFINITY) continue;
    const float f = m == -INFINITY ? 0.f : exp2f(m - mn);
    l *= f;
#pragma unroll
    for (int e = 0; e < 4; ++e) acc[e] *= f;
    m = mn;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (a[u].x == -INFINITY) continue;
      const float w = exp2f(a[u].x - m);
      l = fmaf(a[u].y, w, l);
      acc[0] = fmaf(v[u].x, w, acc[0]);
      acc[1] = fmaf(v[u].y, w, acc[1]);
      acc[2] = fmaf(v[u].z, w, acc[2]);
      acc[3] = fmaf(v[u].w, w, acc[3]);
    }
  }
  RowOut<T, D, BR>(p, po, r, m, l, d == 0).put(d, acc);
}

// ---- host side ---------------------------------------------------------------------

template <typename T, int D, int BR>
mgqa_status launch_merge(const CacheAttnParams &p, int grid, cudaStream_t s) {
  const int blocks = p.by_unit ? p.B * p.Hkv * p.RB : grid;
  const dim3 g((unsigned)blocks, (std::min(p.block_rows, p.R) + 15) / 16, D / 32);
  const cudaError_t e = launch_pdl(cache_merge_kernel<T, D, BR>, g, dim3(kMergeThreads), 0, s, p);
  if (e != cudaSuccess) return fail(MGQA_ERR_CUDA, "cache attention merge launch: %s", cudaGetErrorString(e));
  return MGQA_OK;
}
template <typename T, int D>
mgqa_status launch_merge(const CacheAttnParams &p, int block_rows, int grid, cudaStream_t s) {
  if (block_rows == 16) return launch_merge<T, D, 16>(p, grid, s);
  if (block_rows == 32) return launch_merge<T, D, 32>(p, grid, s);
  if (block_rows == 64) return launch_merge<T, D, 64>(p, grid, s);
  if constexpr (sizeof(T) == 4) {
    if (block_rows == 4) return launch_merge<T, D, 4>(p, grid, s);
    if (block_rows == 8) return launch_merge<T, D, 8>(p, grid, s);
    if (block_rows == 48) return launch_merge<T, D, 48>(p, grid, s);
  } else {
    if (block_rows == 128) return launch_merge<T, D, 128>(p, grid, s);
    if (block_rows == 256) return launch_merge<T, D, 256>(p, grid, s);
  }
  return fail(MGQA_ERR_UNSUPPORTED, "merge: blocks of %d rows", block_rows);
}

}  // namespace

size_t cache_attn_workspace_bytes() {
  // two partial results per CTA, rows of D + 2 floats: up to 128 rows with two
  // CTAs an SM, up to 256 with one; and a word about every run's end
  return kCacheAttnMaxCtas * sizeof(int4) + (size_t)kCacheAttnMaxCtas / 2 * 2 * 256 * (128 + 2) * sizeof(float);
}

mgqa_status launch_cache_merge(const CacheAttnParams &p, mgqa_dtype dt, int D, int block_rows, int grid,
                               cudaStream_t s) {
  if (dt == MGQA_BF16)
    return D == 64 ? launch_merge<__nv_bfloat16, 64>(p, block_rows, grid, s)
                   : launch_merge<__nv_bfloat16, 128>(p, block_rows, grid, s);
  if (dt == MGQA_FP16)
    return D == 64 ? launch_merge<__half, 64>(p, block_rows, grid, s) : launch_merge<__half, 128>(p, block_rows, grid, s);
  return D == 64 ? launch_merge<float, 64>(p, block_rows, grid, s) : launch_merge<float, 128>(p, block_rows, grid, s);
}

mgqa_status launch_cache_attn(const mgqa_args &a, const mgqa_pages *pages, const mgqa_tree *tree, int32_t window,
                              int32_t sinks, void *ws, cudaStream_t s) {
  CacheAttnParams p{};
  p.q = a.q; p.k = a.k; p.v = a.v; p.out = a.out;
  for (int t = 0; t < 3; ++t) {
    p.qs[t] = a.q_stride[t]; p.ks[t] = a.k_stride[t];
    p.vs[t] = a.v_stride[t]; p.os[t] = a.o_stride[t];
  }
  p.cap = a.Lk;
  p.page_shift = -1;
  if (pages) {
    p.table = pages->table;
    p.table_stride = pages->table_stride;
    p.page_size = pages->page_size;
    p.num_pages = pages->num_pages;
    if ((p.page_size & (p.page_size - 1)) == 0)
      for (p.page_shift = 0; (1 << p.page_shift) < p.page_size;) ++p.page_shift;
  }
  p.kv_len = a.kv_len;
  p.window = window > 0 ? std::min(window, kNoWindow - 1) : kNoWindow;
  p.sinks = sinks;
  if (tree) {
    p.tree = 1;
    p.kn = tree->k_new; p.vn = tree->v_new;
    for (int t = 0; t < 3; ++t) {
      p.kns[t] = tree->k_stride[t];
      p.vns[t] = tree->v_stride[t];
    }
    p.bits = tree->bits;
    p.bits_b = tree->bits_stride_b;
    p.bits_t = tree->bits_stride_t;
    p.tree_len = tree->len;
  }
  p.B = a.B; p.Hq = a.Hq; p.Hkv = a.Hkv; p.T = a.Lq;
  p.n_rep = a.Hq / a.Hkv;
  p.R = p.T * p.n_rep;
  p.scale_log2 = a.scale * kLog2e;
  p.lse = a.lse; p.err = a.dev_error;
  const CacheAttnLaunch how{ws, device_sm_count()};
  if (how.sms < 1) return fail(MGQA_ERR_CUDA, "cannot read the SM count of the current device");
  if (a.dtype == MGQA_FP32) return launch_cache_attn_f32(p, a.D, how, s);
  if (cache_attn_tma_takes(p, a.dtype, a.D)) return launch_cache_attn_tma(p, a.dtype, a.D, how, s);
  return launch_cache_attn_tc(p, a.dtype, a.D, how, s);
}

}  // namespace mgqa
