// Eviction from a cache by accumulated attention weight. A request with more than
// `budget` slots keeps its first `sinks` and its last `recent` ones and, of each
// layer's and KV head's others, the budget - sinks - recent of the largest weight
// (of equal ones the first; a NaN is less than any number), in their order, in slots
// 0 .. budget - 1; the weights move along, and those of the slots given up become 0.
//
//   select -- a block per (layer, request, KV head): the smallest weight that stays,
//             by three passes over the weights as ordered integers (11, 11 and 10
//             bits, counted in shared memory), then one pass that writes the kept
//             slots, in order, to the workspace and the weights to their new places.
//   move   -- the rows, in place. Every row moves towards the front, so rounds of
//             consecutive rows, each read as a whole before any of it is written,
//             overwrite nothing that a later round reads. A cluster of up to 16
//             blocks takes a (layer, request, KV head) and a barrier parts a round's
//             reads from its writes. Rows are read past the L1, which another block
//             of the launch writes to.
//   free   -- with counts of the pages: the table entries behind the budget go.
// The kept rows are read once and written once: that is the floor, and the weights
// twice.
#include <algorithm>

#include "common.cuh"
#include "internal.h"

namespace mgqa {
namespace {

constexpr int kSelectThreads = 1024;
constexpr int kBins = 2048;

struct EvictParams {
  char *k, *v;
  int64_t ks[4], vs[4];  // layer, page, head, slot strides in bytes
  int32_t layers, num_pages, Hkv, page_size, pieces, rows, max_pages;
  int32_t *table;
  int64_t table_stride;
  const int32_t *kv_len;
  int32_t *ref, *err, *kv_len_out;
  const float *w;
  float *w_out;
  int64_t wi[3], wo[3];  // layer, request, head strides of the weights
  int32_t slots;  // of a request that there are weights for, too
  int32_t budget, sinks, recent;
  int32_t *plan;   // [rows]: 1: the request is cut to the budget
  int32_t *kept;   // [layers][rows][Hkv][budget] slots that stay
  int32_t cluster;
};

// A weight as an integer of the same order (NaN lowest, one zero).
MGQA_DEV uint32_t ordered(float x) {
  uint32_t u = __float_as_uint(x);
  if ((u & 0x7fffffffu) > 0x7f800000u) return 0u;
  if (u == 0x80000000u) u = 0u;
  return u >> 31 ? ~u : u | 0x80000000u;
}

// Exclusive prefix sum over the block; *total receives the sum. scratch: 33 ints.
MGQA_DEV int block_scan(int x, int *scratch, int *total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int inc = x;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int up = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += up;
  }
  if (lane == 31) scratch[warp] = inc;
  __syncthreads();
  if (warp == 0) {
    const int w = scratch[lane];
    int wi = w;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int up = __shfl_up_sync(0xffffffffu, wi, o);
      if (lane >= o) wi += up;
    }
    scratch[lane] = wi - w;
    if (lane == 31) scratch[32] = wi;
  }
  __syncthreads();
  const int r = scratch[warp] + inc - x;
  *total = scratch[32];
  __syncthreads();
  return r;
}

__global__ void __launch_bounds__(kSelectThreads)
evict_select_kernel(const __grid_constant__ EvictParams p) {
  __shared__ int bins[kBins];
  __shared__ int scratch[33];
  __shared__ uint32_t s_digit;
  __shared__ int s_left;
  const int tid = threadIdx.x;
  const int g = blockIdx.x % p.Hkv, b = blockIdx.x / p.Hkv % p.rows, layer = blockIdx.x / p.Hkv / p.rows;
  grid_dependency_wait();
  allow_dependents();
  const int n = __ldcg(p.kv_len + b);
  const bool first = layer == 0 && g == 0;
  bool bad = n < 0 || n > p.slots;
  if (!bad && n > p.budget && p.table) {  // every page that is read is there, and none that is written is shared
    const int np = (n + p.page_size - 1) / p.page_size, wp = (p.budget + p.page_size - 1) / p.page_size;
    int wrong = 0;
    for (int i = tid; i < np; i += kSelectThreads) {
      const int e = __ldcg(p.table + (int64_t)b * p.table_stride + i);
      if ((unsigned)e >= (unsigned)p.num_pages || (p.ref && i < wp && __ldcg(p.ref + e) > 1)) wrong = 1;
    }
    bad = __syncthreads_or(wrong) != 0;
  }
  const bool over = !bad && n > p.budget;
  if (first && tid == 0) {
    p.plan[b] = over;
    if (bad) report_error(p.err, MGQA_ERR_INVALID_ARG);
  }
  const float *w = p.w + layer * p.wi[0] + b * p.wi[1] + g * p.wi[2];
  float *out = p.w_out + layer * p.wo[0] + b * p.wo[1] + g * p.wo[2];
  if (!over) {
    if (out != w && !bad)
      for (int j = tid; j < n; j += kSelectThreads) out[j] = __ldcg(w + j);
    return;
  }
  // ---- the weight of rank `left` among slots [from, to)
  const int from = p.sinks, to = n - p.recent;
  int left = p.budget - p.sinks - p.recent;  // how many of them stay
  uint32_t cut = 0xffffffffu;                // everything above it stays, and `left` of those equal to it
  if (left > 0) {
    cut = 0u;
    for (int pass = 0; pass < 3; ++pass) {
      const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0, width = pass == 2 ? 10 : 11;
      const int high = shift + width;
      for (int i = tid; i < kBins; i += kSelectThreads) bins[i] = 0;
      __syncthreads();
      for (int j = from + tid; j < to; j += kSelectThreads) {
        const uint32_t u = ordered(__ldcg(w + j));
        if (pass == 0 || u >> high == cut >> high) atomicAdd(&bins[u >> shift & ((1u << width) - 1u)], 1);
      }
      __syncthreads();
      // bins from the top: thread t has bins 2047 - 2 t and 2046 - 2 t
      const int hi = bins[kBins - 1 - 2 * tid], lo = bins[kBins - 2 - 2 * tid];
      int total;
      const int above = block_scan(hi + lo, scratch, &total);
      if (above < left && above + hi + lo >= left) {
        const bool top = above + hi >= left;
        s_digit = (uint32_t)(kBins - (top ? 1 : 2) - 2 * tid);
        s_left = left - above - (top ? 0 : hi);
      }
      __syncthreads();
      cut |= s_digit << shift;
      left = s_left;
      __syncthreads();
    }
  }
  // ---- the kept slots in order, and their weights
  int32_t *kept = p.kept + (int64_t)blockIdx.x * p.budget;
  int sure = 0, equal = 0;  // kept for sure, and equal to the cut, ahead of this round
  for (int j0 = 0; j0 < n; j0 += 4 * kSelectThreads) {
    float x[4];
    int mine = 0;
    uint32_t what = 0u;  // 2 bits a slot: 1 kept, 2 equal
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int j = j0 + 4 * tid + i;
      if (j < n) {
        x[i] = __ldcg(w + j);
        const uint32_t u = ordered(x[i]);
        const bool keep = j < from || j >= to || (left > 0 && u > cut);
        const bool same = !keep && left > 0 && u == cut;
        mine += keep ? 1 : same ? 1 << 16 : 0;
        what |= (keep ? 1u : same ? 2u : 0u) << (2 * i);
      }
    }
    int total;
    const int ahead = block_scan(mine, scratch, &total);  // (its barriers: the round's weights have been read)
    int a = sure + (ahead & 0xffff), e = equal + (ahead >> 16);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t k = what >> (2 * i) & 3u;
      if (k == 1u || (k == 2u && e < left)) {
        const int d = a + min(e, left);
        kept[d] = j0 + 4 * tid + i;
        out[d] = x[i];
      }
      a += k == 1u;
      e += k == 2u;
    }
    sure += total & 0xffff;
    equal += total >> 16;
  }
  __syncthreads();
  for (int j = p.budget + tid; j < n; j += kSelectThreads) out[j] = 0.f;
}

constexpr int kMoveThreads = 512;
constexpr int kMoveU = 4;  // 16-byte pieces of K, and of V, that a thread holds

__global__ void __launch_bounds__(kMoveThreads, 2)
evict_move_kernel(const __grid_constant__ EvictParams p) {
  const int tid = threadIdx.x, C = p.cluster;
  const int unit = blockIdx.x / C, rank = blockIdx.x % C;
  const int g = unit % p.Hkv, b = unit / p.Hkv % p.rows, layer = unit / p.Hkv / p.rows;
  grid_dependency_wait();
  allow_dependents();
  const bool over = __ldcg(p.plan + b);
  if (unit % p.Hkv == 0 && layer == 0 && rank == 0 && tid == 0)
    p.kv_len_out[b] = over ? p.budget : __ldcg(p.kv_len + b);
  if (!over) return;  // (the whole cluster)
  const int32_t *kept = p.kept + (int64_t)unit * p.budget;
  char *k = p.k + layer * p.ks[0] + (int64_t)g * p.ks[2], *v = p.v + layer * p.vs[0] + (int64_t)g * p.vs[2];
  const auto place = [&](int j, int64_t &ok, int64_t &ov) {  // of slot j
    int page = b, slot = j;
    if (p.table) {
      const int i = j / p.page_size;
      page = __ldcg(p.table + (int64_t)b * p.table_stride + i);
      slot = j - i * p.page_size;
    }
    ok = (int64_t)page * p.ks[1] + (int64_t)slot * p.ks[3];
    ov = (int64_t)page * p.vs[1] + (int64_t)slot * p.vs[3];
  };
  const int64_t all = (int64_t)p.budget * p.pieces, step = (int64_t)kMoveThreads * kMoveU * C;
  for (int64_t i0 = 0; i0 < all; i0 += step) {
    uint4 x[kMoveU], y[kMoveU];
    int64_t tk[kMoveU], tv[kMoveU];  // where to; -1: nowhere
#pragma unroll
    for (int u = 0; u < kMoveU; ++u) {
      const int64_t i = i0 + ((int64_t)u * C + rank) * kMoveThreads + tid;
      tk[u] = -1;
      tv[u] = 0;
      if (i < all) {
        const int d = (int)(i / p.pieces), piece = (int)(i - (int64_t)d * p.pieces) * 16;
        const int j = __ldcg(kept + d);
        if (j != d) {
          int64_t fk, fv;
          place(j, fk, fv);
          place(d, tk[u], tv[u]);
          tk[u] += piece;
          tv[u] += piece;
          x[u] = __ldcg(reinterpret_cast<const uint4 *>(k + fk + piece));
          y[u] = __ldcg(reinterpret_cast<const uint4 *>(v + fv + piece));
        }
      }
    }
    if (C > 1) cluster_sync();
    else __syncthreads();
#pragma unroll
    for (int u = 0; u < kMoveU; ++u)
      if (tk[u] >= 0) {
        __stcg(reinterpret_cast<uint4 *>(k + tk[u]), x[u]);
        __stcg(reinterpret_cast<uint4 *>(v + tv[u]), y[u]);
      }
  }
}

__global__ void __launch_bounds__(256) evict_free_kernel(const __grid_constant__ EvictParams p) {
  const int b = blockIdx.x;
  grid_dependency_wait();
  allow_dependents();
  if (!__ldcg(p.plan + b)) return;
  for (int i = (p.budget + p.page_size - 1) / p.page_size + (int)threadIdx.x; i < p.max_pages; i += 256) {
    int32_t *at = p.table + (int64_t)b * p.table_stride + i;
    const int e = __ldcg(at);
    if ((unsigned)e < (unsigned)p.num_pages) atomicSub(p.ref + e, 1);
    *at = -1;
  }
}

int64_t aligned16(int64_t n) { return (n + 15) / 16 * 16; }

}  // namespace

size_t cache_evict_workspace_bytes(const mgqa_cache &c, int32_t budget) {
  return (size_t)(aligned16((int64_t)c.rows * 4) + aligned16((int64_t)c.layers * c.rows * c.Hkv * budget * 4));
}

mgqa_status launch_cache_evict(const mgqa_cache &c, const float *weight, const int64_t *in, float *weight_out,
                               const int64_t *out, int32_t weight_slots, int32_t budget, int32_t sinks, int32_t recent,
                               int32_t *kv_len_out, void *ws, cudaStream_t s) {
  EvictParams p{};
  const int64_t es = c.dtype == MGQA_FP32 ? 4 : 2;
  p.k = static_cast<char *>(c.k);
  p.v = static_cast<char *>(c.v);
  for (int t = 0; t < 4; ++t) {
    p.ks[t] = c.k_stride[t] * es;
    p.vs[t] = c.v_stride[t] * es;
  }
  p.layers = c.layers; p.num_pages = c.num_pages; p.Hkv = c.Hkv; p.page_size = c.page_size;
  p.pieces = (int32_t)(c.D * es / 16);
  p.rows = c.rows; p.max_pages = c.max_pages;
  p.table = c.page_table; p.table_stride = c.table_stride;
  p.kv_len = c.kv_len; p.ref = c.ref; p.err = c.dev_error; p.kv_len_out = kv_len_out;
  p.w = weight; p.w_out = weight_out;
  for (int t = 0; t < 3; ++t) {
    p.wi[t] = in[t];
    p.wo[t] = out[t];
  }
  p.slots = (int32_t)std::min<int64_t>(weight_slots, c.page_table ? (int64_t)c.max_pages * c.page_size : c.page_size);
  p.budget = budget; p.sinks = sinks; p.recent = recent;
  p.plan = static_cast<int32_t *>(ws);
  p.kept = reinterpret_cast<int32_t *>(static_cast<char *>(ws) + aligned16((int64_t)c.rows * 4));
  const int sms = device_sm_count();
  if (sms < 1) return fail(MGQA_ERR_CUDA, "cannot read the SM count of the current device");
  const int64_t units = (int64_t)c.layers * c.rows * c.Hkv;
  const int64_t rounds = ((int64_t)budget * p.pieces + kMoveThreads * kMoveU - 1) / (kMoveThreads * kMoveU);
  p.cluster = 1;
  while (p.cluster < 16 && p.cluster < rounds && units * p.cluster * 2 <= 2 * sms) p.cluster *= 2;
  static std::atomic<uint64_t> attr{0};
  mgqa_status st = ensure_cluster_attr(evict_move_kernel, 0, attr, "cache eviction kernel");
  if (st != MGQA_OK) return st;
  cudaError_t e = launch_pdl(evict_select_kernel, dim3((unsigned)units), dim3(kSelectThreads), 0, s, p);
  if (e == cudaSuccess)
    e = launch_pdl_cluster(evict_move_kernel, dim3((unsigned)(units * p.cluster)), dim3(kMoveThreads), 0, s, p.cluster, p);
  if (e == cudaSuccess && p.ref && p.table)
    e = launch_pdl(evict_free_kernel, dim3(c.rows), dim3(256), 0, s, p);
  if (e != cudaSuccess) return fail(MGQA_ERR_CUDA, "cache eviction launch: %s", cudaGetErrorString(e));
  return MGQA_OK;
}

}  // namespace mgqa
