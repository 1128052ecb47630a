// Work split of the cache attention kernels (one new token, or a tree of
// drafted tokens, per request over a cache in slots or pages).
//
// A request's keys are cut into tiles of 2^tile_shift keys: the tiles of absolute
// cache slots that some query of the request may see (the sinks' tiles, then
// the window's), then the tiles of its drafted tokens. A unit is one (request,
// KV head, block of query rows) with the request's tiles, ahead of which it
// counts `lead` tiles for what a unit costs besides (its query rows, its
// results, the pipeline's fill). The units form one long row of tiles, which
// the CTAs cut into equal runs. Rows of very different lengths so cost every
// CTA the same, whatever the batch. A unit inside one run is finished by its
// CTA; a unit that crosses a run's end leaves one partial result per run in the
// workspace, and the merge kernel joins them in ascending order. The cut depends
// on the lengths, the call's shapes and the device alone, so results repeat bit
// for bit.
#pragma once

#include "common.cuh"
#include "internal.h"

namespace mgqa {

constexpr int kTile = 64;  // keys of a tile (but for the tensor-memory kernel's larger form)
constexpr int kMaxDrafts = kMaxDraftsHost;
constexpr int kNoWindow = 1 << 30;

struct CacheAttnParams {
  const void *q, *k, *v, *kn, *vn;
  void *out;
  int64_t qs[3], ks[3], vs[3], kns[3], vns[3], os[3];  // (batch | page, head, position | slot)
  const int32_t *table;  // [B][max_pages], null: the static cache (one page per request)
  int64_t table_stride;
  int32_t page_size, page_shift;  // page_shift: log2 of a power-of-two page_size, else -1
  int32_t num_pages, cap;         // cap: slots of a request
  const int32_t *kv_len, *tree_len;
  const uint32_t *bits;  // null: each draft sees those before it
  int64_t bits_b, bits_t;
  int32_t window, sinks;  // window: kNoWindow when there is none
  int32_t tree;           // 1: drafts follow the cache; 0: the queries are the last T cached tokens
  int32_t B, Hq, Hkv, T, n_rep, R, RB;  // R = T * n_rep rows per KV head, in RB blocks
  int32_t block_rows;                   // query rows of a block (a unit's)
  int32_t tile_shift;                   // log2 of a tile's keys
  int32_t lead;                         // tiles counted for a unit's own cost
  int32_t min_run;                      // fewest tiles of a CTA's run
  float scale_log2;
  float *lse;
  int32_t *err;
  float *part_o;    // [2 * grid][D / 4][block rows][4] unnormalised partial outputs
  float2 *part_ml;  // [2 * grid][block rows] their (max, sum)
  // What the merge kernel has to join: (request, unit, last run (-1: nothing),
  // first run). By unit when there are no more units than runs, else by the run
  // that ends with a unit's first piece.
  int4 *cuts;
  int32_t by_unit, grid;
};

// What every launcher of the cache attention needs besides the parameters.
struct CacheAttnLaunch {
  void *workspace;
  int sms;
};

// Tiles of one unit (a request's keys), at most.
inline int64_t most_tiles(const CacheAttnParams &p) {
  const int64_t tile = (int64_t)1 << p.tile_shift;
  const int64_t span = (int64_t)p.window + p.T + p.sinks + 4 * tile;
  const int64_t keys = p.cap < span ? p.cap : span;
  return (keys + tile - 1) / tile + 2 + (p.T + tile - 1) / tile;
}

// The workspace as the partial results of `grid` CTAs (two each).
inline void set_partials(CacheAttnParams &p, void *ws, int grid, int block_rows, int D) {
  p.grid = grid;
  p.by_unit = (int64_t)p.B * p.Hkv * p.RB <= grid;
  p.cuts = static_cast<int4 *>(ws);
  p.part_o = reinterpret_cast<float *>(p.cuts + kCacheAttnMaxCtas);
  p.part_ml = reinterpret_cast<float2 *>(p.part_o + (size_t)2 * grid * block_rows * D);
}

// The parameters of a call, but for those of the kernel's form.
void cache_attn_params(const mgqa_args &a, const mgqa_pages *pages, const mgqa_tree *tree, int32_t window,
                       int32_t sinks, CacheAttnParams &p);
mgqa_status launch_cache_merge(const CacheAttnParams &p, mgqa_dtype dt, int D, int block_rows, int grid,
                               cudaStream_t s);
// 16 bits on mma.sync: few rows, or any (in blocks of 64).
bool cache_attn_tma_takes(const CacheAttnParams &p, mgqa_dtype dt, int D);
mgqa_status launch_cache_attn_tma(const CacheAttnParams &p, mgqa_dtype dt, int D, const CacheAttnLaunch &how,
                                  cudaStream_t s);
// fp32 on the CUDA cores.
mgqa_status launch_cache_attn_f32(const CacheAttnParams &p, int D, const CacheAttnLaunch &how, cudaStream_t s);
// 16 bits in tensor memory, for more rows.
bool cache_attn_tc_takes(const CacheAttnParams &p);
mgqa_status launch_cache_attn_tc(const CacheAttnParams &p, mgqa_dtype dt, int D, const CacheAttnLaunch &how,
                                 cudaStream_t s);
// Tensor maps of the cache (boxes of `box_rows` slots: the largest power of two
// up to `tile` that divides the page) and of the drafts; box_rows 0: the call is
// fetched row by row, without maps.
bool cache_attn_maps(const CacheAttnParams &p, mgqa_dtype dt, int D, int tile, CUtensorMap (&maps)[4], int &box_rows);

// What one request's queries may see.
struct RowPlan {
  int n;        // cached tokens
  int live;     // drafted tokens
  int lo;       // first slot of the window (of the query that reaches furthest back)
  int s_end;    // sinks in front of it: [0, s_end)
  int ns, mt0;  // sink tiles; the window's tiles start at tile mt0
  int np, nt;   // tiles of cached keys; all tiles (at least one, which may be empty)
};

MGQA_DEV RowPlan plan_row(const CacheAttnParams &p, int b, bool report) {
  RowPlan r;
  int n = __ldg(p.kv_len + b);
  int live = p.tree ? p.T : 0;
  bool bad = n < 0 || n > p.cap;
  if (p.tree_len) {
    live = __ldg(p.tree_len + b);
    bad = bad || live < 0 || live > p.T;
    live = min(max(live, 0), p.T);
  }
  if (bad && report) report_error(p.err, MGQA_ERR_INVALID_ARG);
  n = min(max(n, 0), p.cap);
  r.n = n;
  r.live = live;
  const int p0 = p.tree ? n : n - p.T;  // the first query's position
  r.lo = min(max(p0 - p.window + 1, 0), n);
  r.s_end = min(p.sinks, r.lo);
  const int ts = p.tile_shift, up = (1 << ts) - 1;
  r.ns = (r.s_end + up) >> ts;
  r.mt0 = max(r.lo >> ts, r.ns);
  r.np = r.ns + (r.lo < n ? max(0, ((n + up) >> ts) - r.mt0) : 0);
  if (p.tree && live == 0) r.np = 0;  // no query is left to see anything
  r.nt = max(1, r.np + ((live + up) >> ts));
  return r;
}

// Brings the kernel's parameters into the constant cache, ahead of the grid-
// dependency wait (each line's first use would cost a miss behind it).
template <typename P>
MGQA_DEV void touch_params(const P &p, int lane) {
  uint32_t x = 0u;
  for (int i = lane; i < (int)(sizeof(P) / 64); i += 32) x ^= reinterpret_cast<const uint32_t *>(&p)[i * 16];
  asm volatile("" ::"r"(x));
}

// The cut of one call: tiles in all, and tiles of a run.
struct Cut {
  int64_t total;
  int64_t run;
};

// a / b for 0 <= a, 0 < b: in 32 bits wherever it fits.
MGQA_DEV int64_t div_up(int64_t a, int b) {
  a += b - 1;
  return a <= 0x7fffffff ? (int64_t)((uint32_t)a / (uint32_t)b) : a / b;
}
MGQA_DEV int div_small(int64_t a, int64_t b) {  // the quotient fits in 32 bits
  return a <= 0x7fffffff && b <= 0x7fffffff ? (int)((uint32_t)a / (uint32_t)b) : (int)(a / b);
}

// Scans the requests (every thread of the block takes part), finds the cut and
// the request that holds the first tile of run `cta`.
struct Located {
  Cut cut;
  int b;          // the request
  int64_t start;  // flat index of its first (lead) tile
  RowPlan rp;     // its plan
};
template <int THREADS>
struct LocateScratch {
  int64_t sum[THREADS / 32];
  int64_t start;
  int32_t b;
  RowPlan rp;
};

template <int THREADS>
MGQA_DEV Located locate(const CacheAttnParams &p, LocateScratch<THREADS> &sc, int grid, int cta, bool report) {
  constexpr int NW = THREADS / 32;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int per = (p.B + THREADS - 1) / THREADS;
  const int64_t units = (int64_t)p.Hkv * p.RB;
  int64_t mine = 0;
  RowPlan one;  // the plan of this thread's only request, when it has one
  one.nt = 0;
  for (int i = 0; i < per; ++i) {
    const int b = tid * per + i;
    if (b < p.B) {
      one = plan_row(p, b, report);
      mine += one.nt + p.lead;
    }
  }
  int64_t inc = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t up = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += up;
  }
  if (lane == 31) sc.sum[warp] = inc;
  __syncthreads();
  int64_t before = 0, total = 0;
#pragma unroll
  for (int w = 0; w < NW; ++w) {
    if (w < warp) before += sc.sum[w];
    total += sc.sum[w];
  }
  before += inc - mine;  // tiles (of one head and row block) of the requests ahead of mine
  Located r;
  r.cut.total = total * units;
  r.cut.run = max((int64_t)p.min_run, div_up(r.cut.total, grid));
  const int64_t want = (int64_t)cta * r.cut.run;
  for (int i = 0; i < per; ++i) {
    const int b = tid * per + i;
    if (b >= p.B) break;
    if (per > 1) one = plan_row(p, b, false);
    const int len = one.nt + p.lead;
    if (want >= before * units && want < (before + len) * units) {
      sc.b = b;
      sc.start = before * units;
      sc.rp = one;
    }
    before += len;
  }
  __syncthreads();
  r.b = sc.b;
  r.start = sc.start;
  r.rp = sc.rp;
  return r;
}

// Page of slot j of a request (-1: no such page; the slot then counts as
// masked and the call reports it).
MGQA_DEV int page_of(const CacheAttnParams &p, int b, int j) {
  if (!p.table) return b;
  const int i = p.page_shift >= 0 ? j >> p.page_shift : j / p.page_size;
  const int pg = __ldg(p.table + (int64_t)b * p.table_stride + i);
  return (unsigned)pg < (unsigned)p.num_pages ? pg : -1;
}
MGQA_DEV int slot_in_page(const CacheAttnParams &p, int j) {
  if (!p.table) return j;
  return p.page_shift >= 0 ? j & (p.page_size - 1) : j % p.page_size;
}

// The drafts' ancestor masks and depths, staged for the masks of a unit:
// see[t] has the bits of the drafts that draft t sees (live ones only), and
// depth[t] the number of other drafts among them.
template <int MAXT>
struct Drafts {
  uint32_t see[MAXT][MAXT / 32];
  int32_t depth[MAXT];
};

template <int MAXT>
MGQA_DEV void stage_drafts(const CacheAttnParams &p, Drafts<MAXT> &d, int b, int live, int tid, int threads) {
  const int W = (p.T + 31) / 32;
  for (int t = tid; t < p.T; t += threads) {
    int depth = 0;
    for (int w = 0; w < W; ++w) {
      uint32_t x = p.bits ? __ldg(p.bits + (int64_t)b * p.bits_b + (int64_t)t * p.bits_t + w)
                          : low_mask(t + 1 - 32 * w);
      x &= low_mask(live - 32 * w);
      if (t >= live) x = 0u;
      d.see[t][w] = x;
      if (t / 32 == w) x &= ~(1u << (t % 32));
      depth += __popc(x);
    }
    d.depth[t] = depth;
  }
}

// Which keys of a partial tile a row may see.
struct RowSight {
  bool ok;    // the row exists and its draft is live
  int t, lo;  // its draft; first slot of its window
};

MGQA_DEV bool sees_cached(const CacheAttnParams &p, const RowSight &rs, int j) {
  return rs.ok && (j >= rs.lo || j < p.sinks);
}
template <int MAXT>
MGQA_DEV bool sees_draft(const CacheAttnParams &p, const Drafts<MAXT> &d, const RowSight &rs, int n, int s) {
  if (!rs.ok || !((d.see[rs.t][s >> 5] >> (s & 31)) & 1u)) return false;
  return n + d.depth[s] >= rs.lo || n + d.depth[s] < p.sinks;
}

// Slot (or draft) of the first key of tile i of a request; kind: 0 cached, 1 drafted.
MGQA_DEV int first_key(const RowPlan &rp, int i, int tile_shift, int &kind) {
  kind = i >= rp.np;
  return (kind ? i - rp.np : (i < rp.ns ? i : rp.mt0 + i - rp.ns)) << tile_shift;
}
// Does key j of that kind count for any query?
MGQA_DEV bool wanted(const RowPlan &rp, int kind, int j) {
  return kind ? j < rp.live : j < rp.n && (j >= rp.lo || j < rp.s_end);
}

// The pieces of a CTA's run, in order: runs of tiles [t0, t1) of one unit.
struct Piece {
  RowPlan rp;
  int b, g, rb, t0, t1;
  int more;  // further runs that the unit reaches into
};
struct Walker {
  int64_t left;  // tiles of the run that are left
  int64_t run;
  int b, unit, v0, units, RB, lead;
  RowPlan rp;

  MGQA_DEV void start(const CacheAttnParams &p, const Located &loc, int cta) {
    const int64_t f = (int64_t)cta * loc.cut.run;
    left = min(loc.cut.run, loc.cut.total - f);
    run = loc.cut.run;
    RB = p.RB;
    lead = p.lead;
    units = p.Hkv * p.RB;
    if (left <= 0) return;
    b = loc.b;
    rp = loc.rp;
    unit = div_small(f - loc.start, rp.nt + lead);
    v0 = (int)(f - loc.start - (int64_t)unit * (rp.nt + lead));
  }
  MGQA_DEV bool next(const CacheAttnParams &p, Piece &pc) {
    while (left > 0) {
      if (unit == units) {
        unit = 0;
        rp = plan_row(p, ++b, false);
      }
      const int v1 = (int)min((int64_t)(rp.nt + lead), v0 + left);
      const int from = v0;
      pc.b = b;
      pc.g = RB == 1 ? unit : unit / RB;
      pc.rb = RB == 1 ? 0 : unit - pc.g * RB;
      left -= v1 - from;
      v0 = 0;
      ++unit;
      if (v1 <= lead) continue;  // the run ends within the unit's lead: the next run has all of it
      pc.rp = rp;
      pc.t0 = max(0, from - lead);
      pc.t1 = v1 - lead;
      pc.more = pc.t1 < rp.nt ? div_small((int64_t)(rp.nt - pc.t1) + run - 1, run) : 0;
      return true;
    }
    return false;
  }
};

// Tells the merge kernel what run `cta` knows (one thread, which walks it too):
// once with `pc` null, then with every piece.
MGQA_DEV void tell_cut(const CacheAttnParams &p, int cta, const Piece *pc) {
  if (!pc) {
    if (!p.by_unit) p.cuts[cta] = make_int4(0, 0, -1, 0);
  } else if (pc->t0 == 0 && (p.by_unit || pc->more)) {
    const int unit = pc->g * p.RB + pc->rb;
    p.cuts[p.by_unit ? pc->b * (p.Hkv * p.RB) + unit : cta] = make_int4(pc->b, unit, pc->more ? cta + pc->more : -1, cta);
  }
}

// Where the finished or partial rows of a piece go. `whole`: the piece is the
// whole unit.
struct PieceOut {
  bool whole;
  int64_t slot;  // partial slot
  int b, g, row0, rows;
};
MGQA_DEV PieceOut out_of(const CacheAttnParams &p, const Piece &pc, int cta) {
  return PieceOut{pc.t0 == 0 && pc.t1 == pc.rp.nt, (int64_t)cta * 2 + (pc.t0 > 0 ? 0 : 1), pc.b, pc.g,
                  pc.rb * p.block_rows, min(p.block_rows, p.R - pc.rb * p.block_rows)};
}

// Where row r of a piece goes: its finished values, or its unnormalised ones.
// BR: rows that a partial result has room for.
template <typename T, int D, int BR>
struct RowOut {
  T *out;       // finished
  float *part;  // else: four features at part, the next four BR * 4 floats on
  float inv;

  // `m`, `l` of the row in log2 units; `tell`: this thread writes what the row
  // has once (its log-sum, or its partial maximum and sum)
  MGQA_DEV RowOut(const CacheAttnParams &p, const PieceOut &po, int r, float m, float l, bool tell) {
    out = nullptr;
    part = nullptr;
    inv = l > 0.f ? 1.f / l : 0.f;
    if (po.whole) {
      const int row = po.row0 + r, t = row / p.n_rep, h = po.g * p.n_rep + row - t * p.n_rep;
      out = static_cast<T *>(p.out) + (int64_t)po.b * p.os[0] + (int64_t)h * p.os[1] + (int64_t)t * p.os[2];
      if (tell && p.lse)
        p.lse[((int64_t)po.b * p.Hq + h) * p.T + t] = l > 0.f ? (m + log2f(l)) * kLn2 : -INFINITY;
    } else {
      part = p.part_o + po.slot * (BR * D) + r * 4;
      if (tell) p.part_ml[po.slot * BR + r] = make_float2(m, l);
    }
  }
  // N consecutive features from d on, unnormalised
  template <int N>
  MGQA_DEV void put(int d, const float (&o)[N]) const {
    static_assert(N == 2 || N == 4 || N == 8, "one store, or two");
    if (part) {
      // (rows side by side: the kernels' lanes hold consecutive rows)
      if constexpr (N == 2) {
        *reinterpret_cast<float2 *>(part + (d / 4) * (BR * 4) + d % 4) = make_float2(o[0], o[1]);
      } else {
#pragma unroll
        for (int i = 0; i < N; i += 4)
          *reinterpret_cast<float4 *>(part + ((d + i) / 4) * (BR * 4)) = make_float4(o[i], o[i + 1], o[i + 2], o[i + 3]);
      }
    } else if constexpr (sizeof(T) == 4) {
      if constexpr (N == 2) {
        *reinterpret_cast<float2 *>(out + d) = make_float2(o[0] * inv, o[1] * inv);
      } else {
#pragma unroll
        for (int i = 0; i < N; i += 4)
          *reinterpret_cast<float4 *>(out + d + i) =
              make_float4(o[i] * inv, o[i + 1] * inv, o[i + 2] * inv, o[i + 3] * inv);
      }
    } else {
      uint32_t w[N / 2];
#pragma unroll
      for (int i = 0; i < N / 2; ++i) w[i] = pack2<T>(o[2 * i] * inv, o[2 * i + 1] * inv);
      if constexpr (N == 2) *reinterpret_cast<uint32_t *>(out + d) = w[0];
      else if constexpr (N == 4) *reinterpret_cast<uint2 *>(out + d) = make_uint2(w[0], w[1]);
      else *reinterpret_cast<uint4 *>(out + d) = make_uint4(w[0], w[1], w[2], w[3]);
    }
  }
};

}  // namespace mgqa
