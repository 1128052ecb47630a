// Warps that stream tiles of a cache's rows into shared memory, each its own, by
// 16-byte asynchronous copies that only it waits for: no barrier between warps inside
// a unit. (One bulk copy per page and tensor, counted on a barrier, took more
// instructions than the products of the 4-bit attention: 918 a tile of 32 keys
// against 665 so, most of them for lanes that issue one after the other.)
#pragma once

#include "cache_producer.cuh"

namespace mgqa {

struct StreamParams {
  TmaParams t;                  // (its strides of k and v are bytes)
  uint32_t kstep[2], vstep[2];  // from page to page and from slot to slot, in 16-byte pieces
  int32_t alike;                // they agree
  int32_t halves;               // 16 slots from a multiple of 16 on lie one after the other
};

// The steps of k and v (null: k's) for rows of `bytes`; false when they are too long.
inline bool set_steps(StreamParams &sp, const int64_t *ks, const int64_t *vs, int bytes, int page_size) {
  for (int t = 0; t < 2; ++t) {
    const int64_t k = ks[2 * t] / 16, v = vs ? vs[2 * t] / 16 : k;
    if (k > 0xffffffffll || v > 0xffffffffll) return false;
    sp.kstep[t] = (uint32_t)k;
    sp.vstep[t] = (uint32_t)v;
  }
  sp.alike = sp.kstep[0] == sp.vstep[0] && sp.kstep[1] == sp.vstep[1];
  sp.halves = sp.alike && sp.kstep[1] == (uint32_t)bytes / 16 && (!sp.t.a.table || page_size % 16 == 0);
  return true;
}

// The tiles of a warp, in order, ahead of their use: every WARPS-th of each piece,
// and each piece PASSES times. What stays the same in a piece is in shared memory, one
// per warp (in registers it took as many as the attention's outputs).
struct alignas(16) Feed {
  int ns, past, np, n;      // first slot of tile t < np: (t < ns ? t : t + past) tiles
  int lo, s_end;            // slots between s_end and lo are hidden
  const int32_t *table;     // of the request; null: static
  const char *k, *v;        // of the KV head (and, static, of the request)
  int t0, pass;
  Pieces pieces;
};

// Where the 16-byte pieces of a row lie within 128 bytes, so that reads meet all banks.
enum Order {
  kAsIs,        // (rows of 80 or 48 bytes: whole rows of eight do so anyway)
  kOddSwapped,  // the halves of odd rows change places: eight lanes read four pieces of two rows
  kXor          // piece ^ row % 8: eight lanes read one piece of eight rows
};

// KEYS rows of P 16-byte pieces a tile, of V too (behind K's) or not.
template <int KEYS, int P, Order ORDER, bool V, int WARPS>
struct Stream {
  static constexpr int TILEB = KEYS * P * 16;  // bytes of a tile of one tensor
  Feed &f;
  int passes;
  int t, end;              // next tile, end of its piece
  int k0, page, slot;      // its first slot; where the lane's row is
  bool want, live;         // the row is wanted; there is a tile

  MGQA_DEV Stream(Feed &feed, int times) : f(feed), passes(times) {}
  MGQA_DEV void settle(const StreamParams &p, int warp, int lane) {  // to the next tile that there is
    const CacheAttnParams &c = p.t.a;
    while (live && t >= end) {
      if (passes > 1 && f.pass + 1 < passes) {
        t = f.t0 + warp;
        __syncwarp();
        if (lane == 0) ++f.pass;
        __syncwarp();
        continue;
      }
      Pieces all = f.pieces;
      Piece pc;
      live = all.next(c, pc);
      __syncwarp();
      if (lane == 0) {
        f.pieces = all;
        f.ns = pc.rp.ns;
        f.past = pc.rp.mt0 - pc.rp.ns;
        f.np = pc.rp.np;
        f.n = pc.rp.n;
        f.lo = pc.rp.lo;
        f.s_end = pc.rp.s_end;
        f.table = c.table ? c.table + (int64_t)pc.b * c.table_stride : nullptr;
        f.k = static_cast<const char *>(c.k) + pc.g * c.ks[1] + (c.table ? 0 : pc.b * c.ks[0]);
        if (V) f.v = static_cast<const char *>(c.v) + pc.g * c.vs[1] + (c.table ? 0 : pc.b * c.vs[0]);
        f.t0 = pc.t0;
        f.pass = 0;
      }
      __syncwarp();
      t = pc.t0 + warp;
      end = pc.t1;
    }
    if (live) {
      const int4 x = *reinterpret_cast<const int4 *>(&f.ns);
      const int2 y = *reinterpret_cast<const int2 *>(&f.lo);
      k0 = (t < x.x ? t : t + x.y) * KEYS;
      const int j = k0 + lane;
      page = slot = 0;
      want = lane < KEYS && t < x.z && j < x.w && (j >= y.x || j < y.y);
      if (want) {
        slot = j;
        if (f.table) {
          const int i = c.page_shift >= 0 ? j >> c.page_shift : j / c.page_size;
          slot = j - i * c.page_size;
          page = __ldg(f.table + i);  // (looked at by the next issue: here its latency would show)
        }
      }
    }
  }
  MGQA_DEV void start(const StreamParams &p, const Pieces &all, int warp, int lane) {
    if (lane == 0) {
      f.pieces = all;
      f.pass = passes;
    }
    __syncwarp();
    live = true;
    t = end = 0;
    settle(p, warp, lane);
  }
  // Starts the copies of the tile that was looked up (zeros for the rows that do not
  // count) and looks the next one up. *what: its first slot and which rows count.
  // Consecutive lanes copy consecutive pieces; a lane knows where its row is.
  MGQA_DEV void issue(const StreamParams &p, int warp, int lane, unsigned char *dst, int2 *what) {
    constexpr int N = KEYS * P / 32;  // copies of a lane
    const bool there = !p.t.a.table || (unsigned)page < (unsigned)p.t.a.num_pages;
    if (want && !there) report_error(p.t.a.err, MGQA_ERR_INVALID_ARG);
    const uint32_t ok = __ballot_sync(0xffffffffu, want && there);
    if (lane == 0) *what = make_int2(k0, (int)ok);
    const uint32_t pg = there ? (uint32_t)page : 0u, sl = (uint32_t)slot;
    const uint64_t at = (uint64_t)pg * p.kstep[0] + (uint64_t)sl * p.kstep[1];  // in pieces
    const char *k = f.k, *v = V ? f.v : nullptr;
    const auto place = [&](int i) {
      const int x = lane + 32 * i;
      return (ORDER == kOddSwapped ? x ^ (x / P & 1) << 2 : ORDER == kXor ? x ^ (x / P & 7) : x) * 16;
    };
    if (p.halves && ok == low_mask(KEYS)) {  // runs of 16 rows
      constexpr int kRun = 16 * P * 16;      // (a lane's piece of the first or the second)
      const uint64_t a = __shfl_sync(0xffffffffu, at, 0), b = __shfl_sync(0xffffffffu, at, 16 % KEYS);
      const char *ka = k + a * 16 + lane * 16, *kb = k + b * 16 + lane * 16 - kRun;
      const char *va = v + a * 16 + lane * 16, *vb = v + b * 16 + lane * 16 - kRun;
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const bool second = 512 * i >= kRun || (512 * i + 512 > kRun && 512 * i + lane * 16 >= kRun);
        cp_async16(dst + place(i), (second ? kb : ka) + 512 * i);
        if (V) cp_async16(dst + TILEB + place(i), (second ? vb : va) + 512 * i);
      }
    } else {
      const uint64_t av = !V || p.alike ? at : (uint64_t)pg * p.vstep[0] + (uint64_t)sl * p.vstep[1];
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const int row = (lane + 32 * i) / P, piece = (lane + 32 * i) % P;
        const uint64_t to = __shfl_sync(0xffffffffu, at, row) + piece;
        const bool take = ok >> row & 1u;
        cp_async16_or_zero(dst + place(i), k + to * 16, take);
        if (V) {
          const uint64_t tv = p.alike ? to : __shfl_sync(0xffffffffu, av, row) + piece;
          cp_async16_or_zero(dst + TILEB + place(i), v + tv * 16, take);
        }
      }
    }
    t += WARPS;
    settle(p, warp, lane);
  }
};

}  // namespace mgqa
