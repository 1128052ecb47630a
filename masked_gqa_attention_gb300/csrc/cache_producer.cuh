// The producer warps (one for K, one for V) of the cache attention kernels: they
// follow the page table and bring every tile into a ring of stages. Two ways:
//   boxes (TMA) that never cross a page, where pages are a multiple of 8 slots. (A
//     box is issued by one lane at a time, ~80 cycles each: with pages of 8 slots
//     one warp for both was slower than the reads.)
//   rows by 16-byte asynchronous copies, for any other page size and for tensors
//     expanded over a dimension (TMA knows no stride of 0): a lane finds where its
//     rows lie, then eight lanes copy a line of 128 bytes of a row, into the boxes'
//     own layout, so the consumers are the same. (Whole rows a pass, with the row's
//     address exchanged for every 16 bytes: 16 trees of 24 drafts 111 us, 105 so; one
//     fp32 row, 64 requests, window 4096, 609 and 418.)
#pragma once

#include <algorithm>

#include "cache_sched.cuh"
#include "tc_ptx.cuh"

namespace mgqa {

struct TmaParams {
  CacheAttnParams a;
  int32_t box_rows;  // slots of a box of cached keys; 0: row by row
  int32_t cluster;   // CTAs of a unit's cluster; 0: equal runs
};

MGQA_DEV uint64_t low64(int n) { return n >= 64 ? ~0ull : (n <= 0 ? 0ull : ((1ull << n) - 1ull)); }

// The pieces of a CTA: its run of the flat tile list, or, in a cluster, its share
// of one unit's tiles.
struct Pieces {
  Walker walk;
  Piece only;
  int S, rank;
  bool first;

  // Every thread of the block (it ends with a barrier).
  template <int THREADS>
  MGQA_DEV void start(const TmaParams &tp, LocateScratch<THREADS> &scratch) {
    const CacheAttnParams &p = tp.a;
    S = tp.cluster;
    rank = S ? (int)blockIdx.x % S : 0;
    first = true;
    if (S) {
      const int unit = (int)blockIdx.x / S, units = p.Hkv * p.RB;
      only.b = unit / units;
      only.g = unit % units / p.RB;
      only.rb = unit % p.RB;
      only.rp = plan_row(p, only.b, rank == 0 && unit % units == 0 && threadIdx.x == 0);
      only.t0 = (int)((int64_t)only.rp.nt * rank / S);
      only.t1 = (int)((int64_t)only.rp.nt * (rank + 1) / S);
      only.more = 0;
      __syncthreads();
    } else {
      walk.start(p, locate<THREADS>(p, scratch, gridDim.x, blockIdx.x, blockIdx.x == 0), blockIdx.x);
    }
  }
  MGQA_DEV bool next(const CacheAttnParams &p, Piece &pc) {
    if (!S) return walk.next(p, pc);
    const bool r = first && only.t0 < only.t1;
    first = false;
    pc = only;
    return r;
  }
  MGQA_DEV bool idle() const { return S && only.t0 >= only.t1; }  // a cluster's CTA without a share
};

// The pages of the boxes of the tiles to come, one a lane of a warp: 32 / NBOX tiles
// with every load, which is started that many tiles ahead (one tile ahead, the
// latency of the page table bounded tiles of 16 KB: 64 rows, D = 64, window 4096,
// 104 us, 99 so).
struct BoxPages {
  int nbox, tiles, base;  // boxes of a tile; tiles of a load; first tile of `now`
  int now, next;          // -2: nothing to fetch, -1: a page that is not there

  MGQA_DEV int look_up(const CacheAttnParams &p, const Piece &pc, int shift, int br, int first) const {
    const int lane = threadIdx.x & 31, t = first + lane / nbox;
    if (t >= pc.t1) return -2;
    const RowPlan &rp = pc.rp;
    int kind;
    const int j0 = first_key(rp, t, shift, kind) + lane % nbox * br;
    const bool some = !kind && j0 < rp.n && ((rp.lo < rp.n && j0 + br > rp.lo) || j0 < rp.s_end);
    return some ? page_of(p, pc.b, j0) : -2;
  }
  MGQA_DEV void start(const CacheAttnParams &p, const Piece &pc, int shift, int br) {
    nbox = (1 << shift) / br;
    tiles = 32 / nbox;
    base = pc.t0;
    now = look_up(p, pc, shift, br, base);
    next = look_up(p, pc, shift, br, base + tiles);
  }
  // The page of box `lane` of tile t (tiles in ascending order).
  MGQA_DEV int page(const CacheAttnParams &p, const Piece &pc, int shift, int br, int t) {
    if (t - base == tiles) {
      base = t;
      now = next;
      next = look_up(p, pc, shift, br, base + tiles);
    }
    const int lane = threadIdx.x & 31;
    const int x = __shfl_sync(0xffffffffu, now, (t - base) * nbox + lane % nbox);
    return lane < nbox ? x : -2;
  }
};

// The rows of one tile of 2^SHIFT keys, for a whole warp. KB boxes of 64, 32 ...
// columns (128 bytes) a row, elements of ES bytes.
template <int KB, int ES, int SHIFT>
struct RowFeed {
  static constexpr int ROWS = 1 << SHIFT, RL = ROWS / 32;  // rows of a tile, of a lane
  int page[RL];  // of this lane's rows of the tile that is issued next (-2: hidden, -1: not there)

  // The pages of tile t, ahead of its issue.
  MGQA_DEV void look_up(const CacheAttnParams &p, const RowPlan &rp, int b, int t) {
    int kind;
    const int k0 = first_key(rp, t, SHIFT, kind) + (int)(threadIdx.x & 31);
#pragma unroll
    for (int s = 0; s < RL; ++s) {
      const int j = k0 + 32 * s;
      page[s] = wanted(rp, kind, j) ? (kind ? b : page_of(p, b, j)) : -2;
    }
  }
  // Starts the copies of the looked-up tile t to dst (boxes of ROWS x 128 bytes,
  // 128-byte swizzled); words: which rows count. The others' rows are left as
  // they are.
  MGQA_DEV void issue(const CacheAttnParams &p, const RowPlan &rp, int g, int t, int of_v, unsigned char *dst,
                      uint32_t (&words)[RL]) const {
    const int lane = threadIdx.x & 31;
    int kind;
    const int k0 = first_key(rp, t, SHIFT, kind);
    const int64_t *st = kind ? (of_v ? p.vns : p.kns) : (of_v ? p.vs : p.ks);
    const char *base = static_cast<const char *>(kind ? (of_v ? p.vn : p.kn) : (of_v ? p.v : p.k));
    const int c = lane & 7;  // 16-byte piece of 128 bytes
#pragma unroll
    for (int s = 0; s < RL; ++s) {
      if (page[s] == -1) report_error(p.err, MGQA_ERR_INVALID_ARG);
      const int j = k0 + 32 * s + lane;
      const int64_t at = (int64_t)page[s] * st[0] + (int64_t)g * st[1] + (int64_t)(kind ? j : slot_in_page(p, j)) * st[2];
      const unsigned long long row = reinterpret_cast<unsigned long long>(base) + (unsigned long long)(at * ES);
      const uint32_t word = words[s] = __ballot_sync(0xffffffffu, page[s] >= 0);
      if (word == 0u) continue;
#pragma unroll
      for (int u = 0; u < 8; ++u) {  // four rows a pass, eight lanes (a line of 128 bytes) each
        const int r = 4 * u + lane / 8;
        const char *src = reinterpret_cast<const char *>(__shfl_sync(0xffffffffu, row, r)) + c * 16;
        if ((word >> r) & 1u)
#pragma unroll
          for (int k = 0; k < KB; ++k)
            cp_async16(dst + k * (ROWS * 128) + (32 * s + r) * 128 + ((c ^ (r & 7)) << 4), src + k * 128);
      }
    }
  }
};

// Arrivals on a stage's full barrier: K's and V's warp, box by box; every lane of
// both when its copies have landed, and K's first lane, row by row.
MGQA_DEV int full_count(const TmaParams &tp) { return tp.box_rows ? 2 : 65; }

// As produce_tiles, row by row.
template <int KB, int COLS, int STAGES>
MGQA_DEV void produce_rows(const TmaParams &tp, Pieces pieces, int of_v, unsigned char *ring, uint2 *ok_words,
                           uint64_t *full, uint64_t *empty) {
  constexpr int TILEB = KB * kTile * 128;
  const CacheAttnParams &p = tp.a;
  const int lane = threadIdx.x & 31;
  RowFeed<KB, 128 / COLS, 6> feed;
  bool ok = true;
  int it = 0;  // tiles started
  Piece pc;
  const bool teller = !of_v && lane == 0 && !pieces.S;
  if (teller) tell_cut(p, blockIdx.x, nullptr);
  while (ok && pieces.next(p, pc)) {
    if (teller) tell_cut(p, blockIdx.x, &pc);
    feed.look_up(p, pc.rp, pc.b, pc.t0);
    for (int t = pc.t0; t < pc.t1; ++t, ++it) {
      const int st = it % STAGES, use = it / STAGES;
      if (use > 0) {
        ok = __all_sync(0xffffffffu, mbar_wait(empty + st, (use - 1) & 1, p.err));
        if (!ok) break;
      }
      const auto now = feed;
      if (t + 1 < pc.t1) feed.look_up(p, pc.rp, pc.b, t + 1);
      uint32_t words[2];
      now.issue(p, pc.rp, pc.g, t, of_v, ring + (st * 2 + of_v) * TILEB, words);
      cp_async_arrive(full + st);
      if (!of_v && lane == 0) {
        ok_words[st] = make_uint2(words[0], words[1]);
        mbar_arrive(full + st);
      }
    }
  }
  cp_async_wait_all();  // no copy may be in flight when the CTA exits
}

// A whole warp, for K (of_v 0) or V. A tile of either in the ring is KB boxes of
// 64 rows x 128 bytes (COLS elements), 128-byte swizzled. Both warps arrive on
// full[stage] (count 2); K's also writes which keys count to ok_words[stage].
template <int KB, int COLS, int STAGES>
MGQA_DEV void produce_tiles(const TmaParams &tp, Pieces pieces, int of_v, const CUtensorMap *tm,
                            const CUtensorMap *tm_new, unsigned char *ring, uint2 *ok_words, uint64_t *full,
                            uint64_t *empty) {
  if (!tp.box_rows) {
    produce_rows<KB, COLS, STAGES>(tp, pieces, of_v, ring, ok_words, full, empty);
    return;
  }
  constexpr int BOXB = kTile * 128, TILEB = KB * BOXB;
  const CacheAttnParams &p = tp.a;
  const int lane = threadIdx.x & 31;
  const int br = tp.box_rows;
  BoxPages pages;
  bool ok = true;
  int it = 0;  // tiles issued
  Piece pc;
  const bool teller = !of_v && lane == 0 && !pieces.S;
  if (teller) tell_cut(p, blockIdx.x, nullptr);
  while (ok && pieces.next(p, pc)) {
    if (teller) tell_cut(p, blockIdx.x, &pc);
    const RowPlan &rp = pc.rp;
    pages.start(p, pc, 6, br);
    for (int t = pc.t0; t < pc.t1 && ok; ++t, ++it) {
      const int page = pages.page(p, pc, 6, br, t);  // (lane i: box i of the tile)
      int kind;
      const int k0 = first_key(rp, t, 6, kind);
      uint64_t bits = 0ull;
      if (kind) {
        bits = lane == 0 ? low64(rp.live - k0) : 0ull;
      } else if (page >= 0) {
        const int j0 = k0 + lane * br;
        bits = (low64(rp.n - j0) & (~low64(rp.lo - j0) | low64(rp.s_end - j0)) & low64(br)) << (lane * br);
      } else if (page == -1) {
        report_error(p.err, MGQA_ERR_INVALID_ARG);
      }
      uint32_t lo = 0u, hi = 0u;
      if (!of_v) {
        lo = __reduce_or_sync(0xffffffffu, (uint32_t)bits);
        hi = __reduce_or_sync(0xffffffffu, (uint32_t)(bits >> 32));
      }
      const bool take = bits != 0ull;
      const int boxes = __popc(__ballot_sync(0xffffffffu, take));
      const int st = it % STAGES, use = it / STAGES;
      if (use > 0) {
        ok = __all_sync(0xffffffffu, mbar_wait(empty + st, (use - 1) & 1, p.err));
        if (!ok) break;
      }
      if (lane == 0) {
        if (!of_v) ok_words[st] = make_uint2(lo, hi);
        mbar_arrive_expect_tx(full + st, (uint32_t)(boxes * (kind ? kTile : br) * 128 * KB));
      }
      __syncwarp();
      if (take) {
        unsigned char *dst = ring + (st * 2 + of_v) * TILEB + (kind ? 0 : lane * br * 128);
        const int slot = kind ? k0 : slot_in_page(p, k0 + lane * br), z = kind ? pc.b : page;
#pragma unroll
        for (int c = 0; c < KB; ++c)
          tc::tma_load_4d(dst + c * BOXB, kind ? tm_new : tm, c * COLS, slot, pc.g, z, full + st);
      }
    }
  }
  // no copy may be in flight when the CTA exits, even if the consumers gave up
  // (the two producers alone arm the full barriers: these are the newest phases)
  __syncwarp();
  for (int i = max(0, it - STAGES); i < it; ++i) mbar_wait(full + i % STAGES, (i / STAGES) & 1, p.err);
}

// The cluster's CTAs join their shares of a unit, each a part of its rows: every
// CTA has its (m, l) in `ml` and its unnormalised rows in `res` (row pitch OP
// floats, 16-byte aligned) of shared memory. The whole block takes part; threads
// [0, WORKERS) do the work.
template <typename T, int D, int ROWS, int OP, int WORKERS>
MGQA_DEV void join_cluster(const CacheAttnParams &p, const Pieces &pieces, const float2 *ml_s, const float *res) {
  __syncwarp();
  cluster_sync();
  const Piece &pc = pieces.only;
  if (threadIdx.x < WORKERS) {
    const PieceOut po{true, 0, pc.b, pc.g, pc.rb * ROWS, min(ROWS, p.R - pc.rb * ROWS)};
    const uint32_t ml0 = smem_u32(ml_s), res0 = smem_u32(res);
    for (int u = pieces.rank * WORKERS + threadIdx.x; u < po.rows * (D / 4); u += pieces.S * WORKERS) {
      const int r = u / (D / 4), d = (u % (D / 4)) * 4;
      float m = -INFINITY, l = 0.f, acc[4] = {0.f, 0.f, 0.f, 0.f};
      float2 ml[16];
      float4 v[16];
#pragma unroll
      for (int x = 0; x < 16; ++x) {  // every load in flight at once
        ml[x] = make_float2(-INFINITY, 0.f);
        v[x] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (x < pieces.S) {
          ml[x] = ld_cluster_f32x2(cluster_map_u32(ml0 + r * 8, x));
          v[x] = ld_cluster_f32x4(cluster_map_u32(res0 + (r * OP + d) * 4, x));
        }
      }
#pragma unroll
      for (int x = 0; x < 16; ++x) m = fmaxf(m, ml[x].x);
#pragma unroll
      for (int x = 0; x < 16; ++x) {
        if (ml[x].x == -INFINITY) continue;
        const float w = exp2f(ml[x].x - m);
        l = fmaf(ml[x].y, w, l);
        acc[0] = fmaf(v[x].x, w, acc[0]);
        acc[1] = fmaf(v[x].y, w, acc[1]);
        acc[2] = fmaf(v[x].z, w, acc[2]);
        acc[3] = fmaf(v[x].w, w, acc[3]);
      }
      RowOut<T, D, ROWS>(p, po, r, m, l, d == 0).put(d, acc);
    }
  }
  __syncwarp();
  cluster_sync();  // no CTA exits while its shared memory is read
}

// Clusters for short calls: whether the reads take at most ~10 us at 6.8 TB/s,
// whatever the lengths are (8 drafts of one request of 4000 tokens over 8 KV heads:
// 15.8 us in a table for 4096 slots, 18.7 as a long call in one for 131072), and how
// many CTAs a unit gets then: no more CTAs than SMs in all (a second one on an SM
// keeps whole clusters waiting).
inline bool short_call(const CacheAttnParams &p, int row_bytes) {
  CacheAttnParams q = p;
  q.tile_shift = 6;
  return (int64_t)p.B * p.Hkv * most_tiles(q) * (2 * kTile * row_bytes) <= (int64_t)64 << 20;
}
inline int cluster_size(const CacheAttnParams &p, int row_bytes, int sms) {
  if (!short_call(p, row_bytes)) return 0;
  const int64_t units = (int64_t)p.B * p.Hkv * p.RB, tiles = most_tiles(p);
  int s = 1;
  while (s < 16 && s < tiles && units * s * 2 <= sms) s *= 2;
  return s;
}

// Short calls leave SMs idle, so a unit's rows go in smaller blocks (half of
// `rows`, and again, down to `least`) while the clusters of all units stay as
// large and fit on the SMs: a block's CTAs read the same keys, from the L2, but
// each has less to compute.
inline int short_block(const CacheAttnParams &p, int row_bytes, int sms, int rows, int least) {
  if (!short_call(p, row_bytes)) return rows;
  CacheAttnParams q = p;
  q.tile_shift = 6;
  auto ctas = [&](int r) { return (int64_t)p.B * p.Hkv * ((p.R + r - 1) / r) * std::min<int64_t>(16, most_tiles(q)); };
  while (rows > least && ctas(rows / 2) <= sms) rows /= 2;
  return rows;
}

}  // namespace mgqa
