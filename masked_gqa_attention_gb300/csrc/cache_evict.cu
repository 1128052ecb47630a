// Eviction from a cache by accumulated attention weight. A request with more than
// `budget` slots keeps its first `sinks` and its last `recent` ones and, of each
// layer's and KV head's others, the budget - sinks - recent of the largest weight
// (of equal ones the first; a NaN is less than any number), in their order, in slots
// 0 .. budget - 1; the weights move along, and those of the slots given up become 0.
//
//   select -- a cluster of 1 to 8 blocks per (layer, request, KV head), each with a
//             part of its weights in shared memory: the smallest weight that stays, by
//             up to three passes over the weights as ordered integers (11, 11 and 10
//             bits, counted per block and summed over the cluster), done when every
//             weight left stays; then the kept slots, in order, to the workspace and
//             the weights to their new places.
//   move   -- the rows, in place. Every row moves towards the front, so rounds of
//             consecutive rows, each read as a whole before any of it is written,
//             overwrite nothing that a later round reads. A cluster of up to 16
//             blocks takes a (layer, request, KV head) and a barrier parts a round's
//             reads from its writes. Rows are read past the L1, which another block
//             of the launch writes to.
//   free   -- with counts of the pages: the table entries behind the budget go.
// The kept rows are read once and written once: that is the floor, and the weights
// twice. (4 layers, 16 requests of 4288 slots on average cut to 2048, 8 heads of 128:
// 175 us, 0.69 of the copy rate: kept rows are 256 bytes here and there, and a block
// reads or writes, not both; records in 4 bits 97. One prompt of 32768 cut to 4096: 30 us,
// 5 of them copies, most of the rest the selection's passes, a cluster barrier and a read
// of eight blocks' counts each; with weights within 0.4 % of one another 31, all equal 28
// (the first slots stay where they are). Rows in registers instead of shared memory: 186
// and 41 us; a selection in one block per head that read its weights for every pass: 49 us
// alone.)
#include <algorithm>

#include "common.cuh"
#include "internal.h"

namespace mgqa {
namespace {

constexpr int kSelectThreads = 512;
constexpr int kSelectWarps = kSelectThreads / 32;
constexpr int kBins = 2048;
constexpr int kPart = 40960;  // weights that a block holds

struct EvictParams {
  char *k, *v;
  int64_t ks[4], vs[4];  // layer, page, head, slot strides in bytes
  int32_t layers, num_pages, Hkv, page_size, page_shift, pieces, rows, max_pages;
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
  int32_t parts;   // blocks of a selection
  int32_t cluster; // blocks of a move
  int32_t round_rows, piece_shift;  // rows of a block's round; of a power of two of pieces, else -1
};

// A weight as an integer of the same order (NaN lowest, one zero).
MGQA_DEV uint32_t ordered(float x) {
  uint32_t u = __float_as_uint(x);
  if ((u & 0x7fffffffu) > 0x7f800000u) return 0u;
  if (u == 0x80000000u) u = 0u;
  return u >> 31 ? ~u : u | 0x80000000u;
}

struct alignas(16) Select {
  int bins[3][kBins];  // one for each pass: none waits for the others to have read it
  int scan[kSelectWarps + 1];
  int2 count[kSelectWarps];  // slots that stay for sure, and those equal to the cut, of a warp's part
  int2 all;                  // of the block, read by its cluster
  uint32_t digit;
  int left, within;
};

// Exclusive prefix sum over the block's threads.
MGQA_DEV int block_scan(int x, int *scan) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int inc = x;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int up = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += up;
  }
  if (lane == 31) scan[warp] = inc;
  __syncthreads();
  int before = 0;
#pragma unroll
  for (int w = 0; w < kSelectWarps; ++w) before += w < warp ? scan[w] : 0;
  return before + inc - x;
}

__global__ void __launch_bounds__(kSelectThreads)
evict_select_kernel(const __grid_constant__ EvictParams p) {
  extern __shared__ __align__(16) float held[];  // the block's weights
  __shared__ Select sm;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, C = p.parts;
  const int unit = blockIdx.x / C, rank = blockIdx.x % C;
  const int g = unit % p.Hkv, b = unit / p.Hkv % p.rows, layer = unit / p.Hkv / p.rows;
  for (int i = tid; i < 3 * kBins; i += kSelectThreads) sm.bins[0][i] = 0;
  grid_dependency_wait();
  allow_dependents();
  const int n = __ldcg(p.kv_len + b);
  const bool first = layer == 0 && g == 0 && rank == 0;
  const bool wrong_n = n < 0 || n > p.slots;
  int wrong = 0;
  // Every page that is read is there, and none that is written is shared (the sinks stay
  // where they are: pages within them are not written).
  if (!wrong_n && n > p.budget && p.table) {
    const int np = (n + p.page_size - 1) / p.page_size, wp = (p.budget + p.page_size - 1) / p.page_size;
    const int w0 = p.sinks / p.page_size;
#pragma unroll 4
    for (int i = tid; i < np; i += kSelectThreads) {
      const int e = __ldcg(p.table + (int64_t)b * p.table_stride + i);
      if ((unsigned)e >= (unsigned)p.num_pages || (p.ref && i >= w0 && i < wp && __ldcg(p.ref + e) > 1))
        wrong = 1;
    }
  }
  const float *w = p.w + layer * p.wi[0] + b * p.wi[1] + g * p.wi[2];
  float *out = p.w_out + layer * p.wo[0] + b * p.wo[1] + g * p.wo[2];
  // a block's part of the slots: whole steps of its warps (beyond what the blocks hold
  // together, the weights are read again for every use, by one block)
  const bool holds = n <= C * kPart;
  if (!holds && rank > 0 && !wrong_n) return;  // (the whole cluster but one, which then uses no cluster barrier)
  const int parts = holds ? C : 1;
  const int part = holds ? (n + C * 32 - 1) / (C * 32) * 32 : n, j0 = rank * part, len = min(part, n - j0);
  const bool want = !wrong_n && n > p.budget;
  if (want && holds) {
    int i = tid;
    for (; i + 7 * kSelectThreads < len; i += 8 * kSelectThreads) {
      float x[8];
#pragma unroll
      for (int u = 0; u < 8; ++u) x[u] = __ldcg(w + j0 + i + u * kSelectThreads);
#pragma unroll
      for (int u = 0; u < 8; ++u) held[i + u * kSelectThreads] = x[u];
    }
#pragma unroll 4
    for (; i < len; i += kSelectThreads) held[i] = __ldcg(w + j0 + i);
  }
  const bool bad = __syncthreads_or(wrong) != 0 || wrong_n;
  const bool over = !bad && want;
  if (first && tid == 0) {
    p.plan[b] = over;
    if (bad) report_error(p.err, MGQA_ERR_INVALID_ARG);
  }
  if (!over) {
    if (out != w && !wrong_n)  // (of a request that is left as it is, too: its length goes on)
      for (int j = rank * kSelectThreads + tid; j < n; j += parts * kSelectThreads) out[j] = __ldcg(w + j);
    return;
  }
  const auto weight = [&](int i) { return holds ? held[i] : __ldcg(w + i); };  // of slot j0 + i

  // ---- the weight of rank `left` among slots [from, to)
  const int from = p.sinks, to = n - p.recent;
  int left = p.budget - p.sinks - p.recent;  // how many of them stay
  uint32_t cut = 0xffffffffu;                // everything above it stays, and `left` of those equal to it,
  int same = 0;                              // compared from this bit on
  if (left > 0) {
    cut = 0u;
    for (int pass = 0; pass < 3; ++pass) {
      const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0, width = pass == 2 ? 10 : 11;
      const int high = shift + width;
      int *bins = sm.bins[pass];
      const int a = max(0, from - j0), z = min(len, to - j0);
#pragma unroll 4
      for (int i = a + tid; i < z; i += kSelectThreads) {
        const uint32_t u = ordered(weight(i));
        if (pass == 0 || u >> high == cut >> high) atomicAdd(&bins[u >> shift & ((1u << width) - 1u)], 1);
      }
      if (parts > 1) cluster_sync();
      else __syncthreads();
      // bins from the top: thread t has bins 2047 - 4 t and the three below
      const int top = kBins - 4 - 4 * tid;
      int4 c = *reinterpret_cast<const int4 *>(bins + top);
      if (parts > 1) {
        float4 f[8];
#pragma unroll
        for (int r = 0; r < 8; ++r) {  // every load in flight at once
          f[r] = make_float4(0.f, 0.f, 0.f, 0.f);
          if (r < parts) f[r] = ld_cluster_f32x4(cluster_map_u32(smem_u32(bins + top), r));
        }
        c = make_int4(0, 0, 0, 0);
#pragma unroll
        for (int r = 0; r < 8; ++r) {
          c.x += __float_as_int(f[r].x);
          c.y += __float_as_int(f[r].y);
          c.z += __float_as_int(f[r].z);
          c.w += __float_as_int(f[r].w);
        }
      }
      const int sum = c.x + c.y + c.z + c.w;
      int above = block_scan(sum, sm.scan);
      if (above < left && above + sum >= left) {
        int at = 3, have = c.w;
        if (above + have < left) { above += have; at = 2; have = c.z; }
        if (above + have < left) { above += have; at = 1; have = c.y; }
        if (above + have < left) { above += have; at = 0; have = c.x; }
        sm.digit = (uint32_t)(top + at);
        sm.left = left - above;
        sm.within = have;
      }
      __syncthreads();
      cut |= sm.digit << shift;
      left = sm.left;
      same = shift;
      if (sm.within == left) break;  // all of them stay
    }
  } else if (parts > 1) {
    cluster_sync();  // every block has its weights: they may be overwritten
  }
  // ---- the kept slots in order, and their weights: a run of the part per warp
  const auto kind = [&](int i, float x) {  // 1: stays, 2: equal to the cut
    const int j = j0 + i;
    const uint32_t u = ordered(x) >> same;
    return j < from || j >= to || (left > 0 && u > cut >> same) ? 1 : left > 0 && u == cut >> same ? 2 : 0;
  };
  const int run = (len + kSelectThreads - 1) / kSelectThreads * 32, i0 = warp * run, i1 = min(len, i0 + run);
  int sure = 0, equal = 0;
  for (int i = i0 + lane; i - lane < i1; i += 32) {
    const int k = i < i1 ? kind(i, weight(i)) : 0;
    sure += __popc(__ballot_sync(0xffffffffu, k == 1));
    equal += __popc(__ballot_sync(0xffffffffu, k == 2));
  }
  if (lane == 0) sm.count[warp] = make_int2(sure, equal);
  __syncthreads();
  sure = equal = 0;
  int2 all = make_int2(0, 0);
  for (int x = 0; x < kSelectWarps; ++x) {
    const int2 c = sm.count[x];
    if (x < warp) {
      sure += c.x;
      equal += c.y;
    }
    all.x += c.x;
    all.y += c.y;
  }
  if (parts > 1) {
    if (tid == 0) sm.all = all;
    cluster_sync();
    float2 f[7];
#pragma unroll
    for (int r = 0; r < 7; ++r) {
      f[r] = make_float2(0.f, 0.f);
      if (r < rank) f[r] = ld_cluster_f32x2(cluster_map_u32(smem_u32(&sm.all), r));
    }
#pragma unroll
    for (int r = 0; r < 7; ++r) {
      sure += __float_as_int(f[r].x);
      equal += __float_as_int(f[r].y);
    }
  }
  int32_t *kept = p.kept + (int64_t)unit * p.budget;
  for (int i = i0 + lane; i - lane < i1; i += 32) {
    const float x = i < i1 ? weight(i) : 0.f;
    const int k = i < i1 ? kind(i, x) : 0;
    const uint32_t ones = __ballot_sync(0xffffffffu, k == 1), twos = __ballot_sync(0xffffffffu, k == 2);
    const uint32_t ahead = low_mask(lane);
    const int e = equal + __popc(twos & ahead), d = sure + __popc(ones & ahead) + min(e, left);
    if (k == 1 || (k == 2 && e < left)) {
      kept[d] = j0 + i;
      if (holds) out[d] = x;
    }
    sure += __popc(ones);
    equal += __popc(twos);
  }
  if (!holds) {  // weights to their places in rounds of the block, each read before it is written
    __syncthreads();
    for (int d0 = 0; d0 < p.budget; d0 += kSelectThreads) {
      const int d = d0 + tid;
      const float x = d < p.budget ? __ldcg(w + kept[d]) : 0.f;
      __syncthreads();
      if (d < p.budget) out[d] = x;
    }
    __syncthreads();
  }
  for (int j = max(p.budget, j0) + tid; j < j0 + len; j += kSelectThreads) out[j] = 0.f;
  if (parts > 1) cluster_sync();  // no block exits while its counts are read
}

constexpr int kMoveThreads = 512;
constexpr int kMoveRows = 256;  // rows of a round, at most

// A row's way, as offsets from the head's K and V; from -1: it stays where it is.
struct Way {
  int64_t from_k, to_k, from_v, to_v;
};
struct alignas(16) Move {
  Way row[2][kMoveRows];  // of a round and of the next one
};

__global__ void __launch_bounds__(kMoveThreads)
evict_move_kernel(const __grid_constant__ EvictParams p) {
  extern __shared__ __align__(16) unsigned char round[];  // a round's rows: K's, then V's
  __shared__ Move sm;
  const int tid = threadIdx.x, C = p.cluster;
  const int unit = blockIdx.x / C, rank = blockIdx.x % C;
  const int g = unit % p.Hkv, b = unit / p.Hkv % p.rows, layer = unit / p.Hkv / p.rows;
  grid_dependency_wait();
  allow_dependents();
  const bool over = __ldcg(p.plan + b);
  if (unit % p.Hkv == 0 && layer == 0 && rank == 0 && tid == 0)
    p.kv_len_out[b] = over ? p.budget : __ldcg(p.kv_len + b);
  if (!over) return;  // (the whole cluster)
  const int32_t *kept = p.kept + (int64_t)unit * p.budget, *table = p.table + (int64_t)b * p.table_stride;
  char *k = p.k + layer * p.ks[0] + (int64_t)g * p.ks[2], *v = p.v + layer * p.vs[0] + (int64_t)g * p.vs[2];
  if (!p.table) {
    k += b * p.ks[1];
    v += b * p.vs[1];
  }
  const auto index = [&](int j) { return p.page_shift >= 0 ? j >> p.page_shift : j / p.page_size; };
  const int R = p.round_rows, step = R * C;
  const auto look = [&](int first, Way *way) {  // rows [first, first + R)
    for (int r = tid; r < R; r += kMoveThreads) {
      const int d = first + r;
      Way x{-1, 0, 0, 0};
      if (d < p.budget) {
        const int j = __ldcg(kept + d);
        if (j != d) {
          int64_t a = 0, b = 0, from = j, to = d;
          if (p.table) {
            a = __ldcg(table + index(j));
            b = __ldcg(table + index(d));
            from = j - index(j) * p.page_size;
            to = d - index(d) * p.page_size;
          }
          x = Way{a * p.ks[1] + from * p.ks[3], b * p.ks[1] + to * p.ks[3], a * p.vs[1] + from * p.vs[3],
                  b * p.vs[1] + to * p.vs[3]};
        }
      }
      way[r] = x;
    }
  };
  // of piece i of a round's K or V
  const auto row_of = [&](int i) { return p.piece_shift >= 0 ? i >> p.piece_shift : i / p.pieces; };
  look(rank * R, sm.row[0]);
  __syncthreads();
  int now = 0;
  for (int d0 = rank * R; d0 < p.budget + rank * R; d0 += step, now ^= 1) {  // (as many rounds for every block)
    const Way *way = sm.row[now];
    const int n = max(0, min(R, p.budget - d0)) * p.pieces;
    unsigned char *round_v = round + R * p.pieces * 16;
#pragma unroll 4
    for (int i = tid; i < n; i += kMoveThreads) {
      const int r = row_of(i), piece = (i - r * p.pieces) * 16;
      if (way[r].from_k < 0) continue;
      cp_async16(round + i * 16, k + way[r].from_k + piece);
      cp_async16(round_v + i * 16, v + way[r].from_v + piece);
    }
    if (d0 + step < p.budget) look(d0 + step, sm.row[now ^ 1]);
    cp_async_wait_all();
    if (C > 1) cluster_sync();
    else __syncthreads();
#pragma unroll 4
    for (int i = tid; i < n; i += kMoveThreads) {
      const int r = row_of(i), piece = (i - r * p.pieces) * 16;
      if (way[r].from_k < 0) continue;
      __stcg(reinterpret_cast<uint4 *>(k + way[r].to_k + piece), *reinterpret_cast<const uint4 *>(round + i * 16));
      __stcg(reinterpret_cast<uint4 *>(v + way[r].to_v + piece), *reinterpret_cast<const uint4 *>(round_v + i * 16));
    }
    __syncthreads();  // the round's rows have been written from shared memory
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


constexpr int kMoveMost = 204800, kMoveBytes = 49152;  // bytes of a block's round: alone on its SM, or not
constexpr int kMoveFill = 4;                         // clusters grow while there are fewer blocks an SM

int64_t aligned16(int64_t n) { return (n + 15) / 16 * 16; }

}  // namespace

size_t cache_evict_workspace_bytes(const mgqa_cache &c, int32_t budget) {
  const int64_t slots = c.page_table ? (int64_t)c.max_pages * c.page_size : c.page_size;
  if (budget >= slots) budget = 0;  // no request is ever cut
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
  p.page_shift = -1;
  if ((c.page_size & (c.page_size - 1)) == 0)
    for (p.page_shift = 0; (1 << p.page_shift) < c.page_size;) ++p.page_shift;
  // more blocks while there are few for the SMs and each has enough to do. (A block is a
  // quarter of an SM's threads. By shared memory three blocks of a move with 64 KB each
  // fit one, and of a selection as few as one with all its weights: large calls take more
  // than one wave.)
  const int row_bytes = p.pieces * 32;  // of K and V
  p.piece_shift = -1;
  if ((p.pieces & (p.pieces - 1)) == 0)
    for (p.piece_shift = 0; (1 << p.piece_shift) < p.pieces;) ++p.piece_shift;
  p.cluster = p.parts = 1;
  const auto fits = [&](int bytes) { return std::max(1, std::min(kMoveRows, bytes / row_bytes)); };
  while (p.cluster < 16 && (int64_t)p.cluster * 64 < budget && units * p.cluster < kMoveFill * sms) p.cluster *= 2;
  p.round_rows = std::min((budget + p.cluster - 1) / p.cluster, fits(units * p.cluster <= sms ? kMoveMost : kMoveBytes));
  if (row_bytes > kMoveMost) return fail(MGQA_ERR_UNSUPPORTED, "cache eviction: rows of more than %d bytes", kMoveMost / 2);
  while (p.parts < 8 && p.slots > p.parts * 8 * kSelectThreads &&
         (units * p.parts < sms || p.slots > p.parts * kPart))
    p.parts *= 2;
  const int held = std::min<int>(kPart, (p.slots + p.parts * 32 - 1) / (p.parts * 32) * 32) * 4;
  static std::atomic<uint64_t> select_attr{0}, move_attr{0};
  mgqa_status st = ensure_cluster_attr(evict_select_kernel, kPart * 4, select_attr, "cache eviction kernel");
  if (st == MGQA_OK) st = ensure_cluster_attr(evict_move_kernel, kMoveMost, move_attr, "cache eviction kernel");
  if (st != MGQA_OK) return st;
  cudaError_t e = launch_pdl_cluster(evict_select_kernel, dim3((unsigned)(units * p.parts)), dim3(kSelectThreads), held, s,
                                     p.parts, p);
  if (e == cudaSuccess)
    e = launch_pdl_cluster(evict_move_kernel, dim3((unsigned)(units * p.cluster)), dim3(kMoveThreads),
                           p.round_rows * row_bytes, s, p.cluster, p);
  if (e == cudaSuccess && p.ref && p.table)
    e = launch_pdl(evict_free_kernel, dim3(c.rows), dim3(256), 0, s, p);
  if (e != cudaSuccess) return fail(MGQA_ERR_CUDA, "cache eviction launch: %s", cudaGetErrorString(e));
  return MGQA_OK;
}

}  // namespace mgqa
