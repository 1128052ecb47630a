// The 16-bit cache attention for up to 64 query rows per KV head (one token's
// heads, or a small tree), and for more in blocks of 64 where tensor memory is
// not used: the formulas of cache_attn.cu.
//
// Reads bound it (64 rows of up to 32768 keys, window 4096: 158 us, 92 % of the
// copy rate; in pages of one slot, row by row, 222). Two producer warps
// (cache_producer.cuh) bring each 64-key tile into a ring of 96 KB, as TMA boxes
// of gcd(page_size, 64) rows x 64 columns, 128-byte swizzled; two CTAs an SM keep
// up to 192 KB in flight. Four consumer warps run the products on mma.sync with no
// block barrier inside a unit: 16 query rows a warp, and with 16 or 32 rows the
// warps take different keys of each tile and join once at the end. (The first
// form, 16-byte copies issued by the consumers themselves, spent ~1200
// instructions a warp and tile, most on addresses: 360 us for 64 paged rows of
// up to 32768 keys, window 4096, where the reads take 148 us.)
//
// Two ways to cut the work, by what the shapes allow at most (the lengths are
// on the device):
//   equal runs (cache_sched.cuh) and a merge kernel, for long calls;
//   a cluster of up to 16 CTAs per unit, for short ones, where the second
//   launch would be a good part of the time: each CTA takes an equal share of
//   the unit's tiles, leaves (m, l, O) in its shared memory, and after a
//   cluster barrier all of them join and write a part of the rows.
#include <algorithm>
#include <cmath>
#include <cstring>

#include "cache_producer.cuh"

namespace mgqa {
namespace {

constexpr int kConsumers = 128;
constexpr int kThreads = kConsumers + 64;

template <int D, int WM>
struct Cfg {
  static constexpr int WK = 4 / WM;      // warps that share a tile's keys
  static constexpr int ROWS = 16 * WM;   // query rows of a CTA
  static constexpr int KW = kTile / WK;  // keys of a warp in a tile
  static constexpr int KB = D / 64;
  static constexpr int BOXB = kTile * 128;
  static constexpr int TILEB = KB * BOXB;        // bytes of a K (or V) tile
  static constexpr int STAGES = 98304 / (2 * TILEB);
  static constexpr int ring = STAGES * 2 * TILEB;
  static constexpr int OP = D + 4;               // row pitch of a CTA's result (floats)
  static_assert(ROWS * OP * 4 <= ring, "a CTA's result fits in the ring");
  struct Misc {
    float join[WK > 1 ? (WK - 1) * WM : 1][16][WK > 1 ? 66 : 1];  // half a result of the warps that join
    float wm[WK][ROWS], wl[WK][ROWS];
    float2 ml[ROWS];  // the CTA's (m, l), read by its cluster
    Drafts<WM == 4 ? kMaxDrafts : 32> drafts;  // (smaller blocks: up to 32)
    LocateScratch<kThreads> scratch;
    uint2 ok[STAGES];  // which keys of a stage's tile count
    uint64_t full[STAGES], empty[STAGES];
    int maxdepth;
  };
  static constexpr int smem = ring + (int)sizeof(Misc) + 1024;
  // byte of 16-byte piece c of row r of a tile (128-byte swizzled boxes of 64 columns)
  static MGQA_DEV uint32_t at(int r, int c) {
    return (uint32_t)((c >> 3) * BOXB + r * 128 + (((c & 7) ^ (r & 7)) << 4));
  }
};

template <typename T, int D, int WM>
__global__ void __launch_bounds__(kThreads, 2)
cache_attn_tma_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                      const __grid_constant__ CUtensorMap tm_kn, const __grid_constant__ CUtensorMap tm_vn,
                      const __grid_constant__ TmaParams tp) {
  using C = Cfg<D, WM>;
  constexpr int WK = C::WK, ROWS = C::ROWS, KW = C::KW, STAGES = C::STAGES;
  const CacheAttnParams &p = tp.a;
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  unsigned char *ring = reinterpret_cast<unsigned char *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
  auto &sm = *reinterpret_cast<typename C::Misc *>(ring + C::ring);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;

  if (tid == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(sm.full + s, full_count(tp));
      mbar_init(sm.empty + s, 4);
    }
    fence_mbarrier_init();
    if (tp.box_rows) {
      tc::prefetch_tensormap(&tm_k);
      tc::prefetch_tensormap(&tm_v);
    }
    if (tp.box_rows && p.tree) {
      tc::prefetch_tensormap(&tm_kn);
      tc::prefetch_tensormap(&tm_vn);
    }
  }
  if (warp == 1) touch_params(tp, lane);
  grid_dependency_wait();
  allow_dependents();  // lengths and tables are final from here on

  Pieces pieces{};
  pieces.start<kThreads>(tp, sm.scratch);  // (its barrier: the mbarriers are initialised)
  const int S = pieces.S;

  if (warp >= 4) {
    const int of_v = warp - 4;
    produce_tiles<C::KB, 64, STAGES>(tp, pieces, of_v, of_v ? &tm_v : &tm_k, of_v ? &tm_vn : &tm_kn, ring, sm.ok,
                                     sm.full, sm.empty);
  } else {
    // ---------------- consumers ----------------
    const int wm = warp / WK, wk = warp % WK;
    const int gq = lane >> 2, tq = lane & 3, mi = lane >> 3, rr = lane & 7;
    bool ok = true;
    int it = 0, staged = -1;
    Piece pc;
    if (pieces.idle() && tid < ROWS) sm.ml[tid] = make_float2(-INFINITY, 0.f);  // no share of the unit
    while (pieces.next(p, pc)) {
      const RowPlan &rp = pc.rp;
      const PieceOut po = out_of(p, pc, blockIdx.x);
      uint32_t qa[D / 16][4];
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        const int row = po.row0 + wm * 16 + gq + 8 * half;
        const bool in = row < p.R;
        const int t = in ? row / p.n_rep : 0, h = pc.g * p.n_rep + (in ? row % p.n_rep : 0);
        const T *src = static_cast<const T *>(p.q) + (int64_t)pc.b * p.qs[0] + (int64_t)h * p.qs[1] + (int64_t)t * p.qs[2];
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          qa[kk][half] = in ? *reinterpret_cast<const uint32_t *>(src + kk * 16 + 2 * tq) : 0u;
          qa[kk][2 + half] = in ? *reinterpret_cast<const uint32_t *>(src + kk * 16 + 8 + 2 * tq) : 0u;
        }
      }
      const bool need_drafts = p.tree && (p.window != kNoWindow || pc.t1 > rp.np);
      if (need_drafts && staged != pc.b) {
        named_sync(1, kConsumers);  // the masks of an earlier request are no longer read
        if (tid == 0) sm.maxdepth = 0;
        stage_drafts(p, sm.drafts, pc.b, rp.live, tid, kConsumers);
        named_sync(1, kConsumers);
        int md = 0;
        for (int x = tid; x < rp.live; x += kConsumers) md = max(md, sm.drafts.depth[x]);
        if (md) atomicMax(&sm.maxdepth, md);
        named_sync(1, kConsumers);
        staged = pc.b;
      }
      RowSight sight[2];
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        const int row = po.row0 + wm * 16 + gq + 8 * half;
        sight[half].t = row / p.n_rep;
        sight[half].ok = row < p.R && (!p.tree || sight[half].t < rp.live);
        const int pt = p.tree ? rp.n + (need_drafts && sight[half].ok ? sm.drafts.depth[sight[half].t] : 0) : rp.n - 1;
        sight[half].lo = pt - p.window + 1;
      }
      // a cached tile behind this slot is inside every row's window
      const int lo_all = rp.n + (p.tree ? (need_drafts ? sm.maxdepth : 0) : -1) - p.window + 1;

      float o[D / 8][4], m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
#pragma unroll
      for (int d = 0; d < D / 8; ++d) o[d][0] = o[d][1] = o[d][2] = o[d][3] = 0.f;

      for (int t = pc.t0; t < pc.t1; ++t, ++it) {
        const int st = it % STAGES;
        if (ok) ok = __all_sync(0xffffffffu, mbar_wait(sm.full + st, (it / STAGES) & 1, p.err));
        if (ok) {
          const unsigned char *kt = ring + st * 2 * C::TILEB, *vt = kt + C::TILEB;
          const uint2 okw = sm.ok[st];
          const int key0 = wk * KW;  // this warp's keys of the tile
          float s[KW / 8][4];
#pragma unroll
          for (int nn = 0; nn < KW / 8; ++nn) s[nn][0] = s[nn][1] = s[nn][2] = s[nn][3] = 0.f;
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk)
#pragma unroll
            for (int np = 0; np < KW / 16; ++np) {
              uint32_t b0, b1, b2, b3;
              ldmatrix_x4(b0, b1, b2, b3, kt + C::at(key0 + np * 16 + (mi >> 1) * 8 + rr, 2 * kk + (mi & 1)));
              mma_16816<T>(s[2 * np], qa[kk][0], qa[kk][1], qa[kk][2], qa[kk][3], b0, b1);
              mma_16816<T>(s[2 * np + 1], qa[kk][0], qa[kk][1], qa[kk][2], qa[kk][3], b2, b3);
            }
          int kind;
          const int k0 = first_key(rp, t, 6, kind);
          const bool clean = (okw.x & okw.y) == 0xffffffffu;
          const bool full = !kind && clean && (k0 >= lo_all || k0 + kTile <= min(p.sinks, rp.s_end));
          if (full) {
#pragma unroll
            for (int nn = 0; nn < KW / 8; ++nn)
#pragma unroll
              for (int e = 0; e < 4; ++e) s[nn][e] *= p.scale_log2;
          } else {
#pragma unroll
            for (int nn = 0; nn < KW / 8; ++nn)
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const int c = key0 + nn * 8 + 2 * tq + (e & 1);
                const RowSight &rs = sight[e >> 1];
                const bool see = ((c < 32 ? okw.x : okw.y) >> (c & 31) & 1u) &&
                                 (kind ? sees_draft(p, sm.drafts, rs, rp.n, k0 + c) : sees_cached(p, rs, k0 + c));
                s[nn][e] = see ? s[nn][e] * p.scale_log2 : -INFINITY;
              }
          }
          float mx[2] = {m[0], m[1]}, mb[2];
#pragma unroll
          for (int nn = 0; nn < KW / 8; ++nn) {
            mx[0] = fmaxf(mx[0], fmaxf(s[nn][0], s[nn][1]));
            mx[1] = fmaxf(mx[1], fmaxf(s[nn][2], s[nn][3]));
          }
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            mx[e] = fmaxf(mx[e], __shfl_xor_sync(0xffffffffu, mx[e], 1));
            mx[e] = fmaxf(mx[e], __shfl_xor_sync(0xffffffffu, mx[e], 2));
            mb[e] = mx[e] == -INFINITY ? 0.f : mx[e];  // nothing seen yet: every weight is 0
          }
          if (__any_sync(0xffffffffu, mx[0] != m[0] || mx[1] != m[1])) {
            const float f0 = fast_exp2(m[0] - mb[0]), f1 = fast_exp2(m[1] - mb[1]);
            l[0] *= f0;
            l[1] *= f1;
#pragma unroll
            for (int d = 0; d < D / 8; ++d) {
              o[d][0] *= f0;
              o[d][1] *= f0;
              o[d][2] *= f1;
              o[d][3] *= f1;
            }
            m[0] = mx[0];
            m[1] = mx[1];
          }
#pragma unroll
          for (int nn = 0; nn < KW / 8; ++nn) {
            s[nn][0] = fast_exp2(s[nn][0] - mb[0]);
            s[nn][1] = fast_exp2(s[nn][1] - mb[0]);
            s[nn][2] = fast_exp2(s[nn][2] - mb[1]);
            s[nn][3] = fast_exp2(s[nn][3] - mb[1]);
            l[0] += s[nn][0] + s[nn][1];
            l[1] += s[nn][2] + s[nn][3];
          }
          // O += P V; P is rounded to the 16-bit type (l keeps the fp32 weights), as
          // the tensor cores' operand: half a step per weight, unbiased over keys
          // (fp16 below 2^-14 of the row's largest weight: 2^-25 of that one).
          // Values of keys that do not count are cleared (their rows may hold anything).
#pragma unroll
          for (int kp = 0; kp < KW / 16; ++kp) {
            const uint32_t a0 = pack2<T>(s[2 * kp][0], s[2 * kp][1]), a1 = pack2<T>(s[2 * kp][2], s[2 * kp][3]);
            const uint32_t a2 = pack2<T>(s[2 * kp + 1][0], s[2 * kp + 1][1]);
            const uint32_t a3 = pack2<T>(s[2 * kp + 1][2], s[2 * kp + 1][3]);
            uint32_t c0 = 0xffffffffu, c1 = 0xffffffffu;
            if (!clean) {
              const int c = key0 + kp * 16 + 2 * tq;  // keys c, c + 1 and c + 8, c + 9
              const uint32_t w = (c < 32 ? okw.x : okw.y) >> (c & 31);
              c0 = (w & 1u ? 0xffffu : 0u) | (w & 2u ? 0xffff0000u : 0u);
              c1 = (w & 0x100u ? 0xffffu : 0u) | (w & 0x200u ? 0xffff0000u : 0u);
            }
#pragma unroll
            for (int dp = 0; dp < D / 16; ++dp) {
              uint32_t b0, b1, b2, b3;
              ldmatrix_x4_trans(b0, b1, b2, b3, vt + C::at(key0 + kp * 16 + (mi & 1) * 8 + rr, 2 * dp + (mi >> 1)));
              mma_16816<T>(o[2 * dp], a0, a1, a2, a3, b0 & c0, b1 & c1);
              mma_16816<T>(o[2 * dp + 1], a0, a1, a2, a3, b2 & c0, b3 & c1);
            }
          }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(sm.empty + st);
      }

      // ---- join the warps that shared the keys
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        l[e] += __shfl_xor_sync(0xffffffffu, l[e], 1);
        l[e] += __shfl_xor_sync(0xffffffffu, l[e], 2);
        if (!sight[e].ok || !ok) {  // scores of a row that sees nothing were never masked in full tiles
          m[e] = -INFINITY;
          l[e] = 0.f;
        }
      }
      if constexpr (WK > 1) {
        float f[2];
        named_sync(1, kConsumers);  // the exchange of an earlier piece has been read
        if (tq == 0) {
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            sm.wm[wk][wm * 16 + gq + 8 * e] = m[e];
            sm.wl[wk][wm * 16 + gq + 8 * e] = l[e];
          }
        }
        named_sync(1, kConsumers);
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int r = wm * 16 + gq + 8 * e;
          float mr = -INFINITY, lr = 0.f;
#pragma unroll
          for (int w = 0; w < WK; ++w) mr = fmaxf(mr, sm.wm[w][r]);
#pragma unroll
          for (int w = 0; w < WK; ++w)
            if (sm.wm[w][r] != -INFINITY) lr = fmaf(sm.wl[w][r], fast_exp2(sm.wm[w][r] - mr), lr);
          f[e] = m[e] == -INFINITY ? 0.f : fast_exp2(m[e] - mr);
          m[e] = mr;
          l[e] = lr;
        }
#pragma unroll
        for (int half = 0; half < D / 64; ++half) {  // 64 features at a time
          if (half) named_sync(1, kConsumers);
#pragma unroll
          for (int d8 = 0; d8 < 8; ++d8) {
            const int d = half * 8 + d8;
#pragma unroll
            for (int e = 0; e < 4; ++e) o[d][e] = f[e >> 1] == 0.f ? 0.f : o[d][e] * f[e >> 1];
            if (wk > 0) {
              float(*dst)[66] = sm.join[(wk - 1) * WM + wm];
              *reinterpret_cast<float2 *>(&dst[gq][d8 * 8 + 2 * tq]) = make_float2(o[d][0], o[d][1]);
              *reinterpret_cast<float2 *>(&dst[gq + 8][d8 * 8 + 2 * tq]) = make_float2(o[d][2], o[d][3]);
            }
          }
          named_sync(1, kConsumers);
          if (wk == 0) {
#pragma unroll
            for (int w = 1; w < WK; ++w)
#pragma unroll
              for (int d8 = 0; d8 < 8; ++d8) {
                const int d = half * 8 + d8;
                const float2 x = *reinterpret_cast<const float2 *>(&sm.join[(w - 1) * WM + wm][gq][d8 * 8 + 2 * tq]);
                const float2 y = *reinterpret_cast<const float2 *>(&sm.join[(w - 1) * WM + wm][gq + 8][d8 * 8 + 2 * tq]);
                o[d][0] += x.x;
                o[d][1] += x.y;
                o[d][2] += y.x;
                o[d][3] += y.y;
              }
          }
        }
      }
      if (!S) {
        if (wk == 0) {
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int r = wm * 16 + gq + 8 * e;
            if (r >= po.rows) continue;
            const RowOut<T, D, ROWS> dst(p, po, r, m[e], l[e], tq == 0);
#pragma unroll
            for (int d = 0; d < D / 8; ++d) {
              const float x[2] = {m[e] == -INFINITY ? 0.f : o[d][2 * e], m[e] == -INFINITY ? 0.f : o[d][2 * e + 1]};
              dst.put(d * 8 + 2 * tq, x);
            }
          }
        }
      } else {
        named_sync(1, kConsumers);  // every tile has been read: the ring takes the CTA's result
        float *res = reinterpret_cast<float *>(ring);
        if (wk == 0) {
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int r = wm * 16 + gq + 8 * e;
            if (tq == 0) sm.ml[r] = make_float2(m[e], l[e]);
#pragma unroll
            for (int d = 0; d < D / 8; ++d)
              *reinterpret_cast<float2 *>(res + r * C::OP + d * 8 + 2 * tq) = make_float2(o[d][2 * e], o[d][2 * e + 1]);
          }
        }
      }
    }
  }

  if (S) join_cluster<T, D, ROWS, C::OP, kConsumers>(p, pieces, sm.ml, reinterpret_cast<const float *>(ring));
}

template <typename T, int D, int WM>
mgqa_status launch_t(const CUtensorMap (&maps)[4], TmaParams tp, const CacheAttnLaunch &how, cudaStream_t s) {
  using C = Cfg<D, WM>;
  auto kern = cache_attn_tma_kernel<T, D, WM>;
  static std::atomic<uint64_t> attr{0};
  mgqa_status st = ensure_cluster_attr(kern, C::smem, attr, "cache attention kernel");
  if (st != MGQA_OK) return st;
  CacheAttnParams &p = tp.a;
  p.block_rows = C::ROWS;
  p.RB = (p.R + C::ROWS - 1) / C::ROWS;
  p.tile_shift = 6;
  const int64_t units = (int64_t)p.B * p.Hkv * p.RB;
  const int64_t tiles = most_tiles(p);  // of one unit, at most
  tp.cluster = cluster_size(p, D * 2, how.sms);
  if (tp.cluster) {
    const cudaError_t e = launch_pdl_cluster(kern, dim3((unsigned)(units * tp.cluster)), dim3(kThreads), C::smem, s,
                                             tp.cluster, maps[0], maps[1], maps[2], maps[3], tp);
    if (e != cudaSuccess) return fail(MGQA_ERR_CUDA, "cache attention launch: %s", cudaGetErrorString(e));
    return MGQA_OK;
  }
  p.lead = 4;
  p.min_run = 4;
  const int grid =
      (int)std::max<int64_t>(1, std::min<int64_t>(std::min(2 * how.sms, kCacheAttnMaxCtas), units * (tiles + p.lead)));
  set_partials(p, how.workspace, grid, C::ROWS, D);
  const cudaError_t e = launch_pdl(kern, dim3(grid), dim3(kThreads), C::smem, s, maps[0], maps[1], maps[2], maps[3], tp);
  if (e != cudaSuccess) return fail(MGQA_ERR_CUDA, "cache attention launch: %s", cudaGetErrorString(e));
  return launch_cache_merge(p, sizeof(T) == 2 && __is_same(T, __half) ? MGQA_FP16 : MGQA_BF16, D, C::ROWS, grid, s);
}

template <typename T, int D>
mgqa_status launch_d(const CUtensorMap (&maps)[4], const TmaParams &tp, const CacheAttnLaunch &how, cudaStream_t s) {
  // the smallest block that holds the rows, or a smaller one on short calls (8 drafts
  // of 16 heads over 2, 4096 slots, D = 128: 10.5 us in blocks of 16 rows, 12.5 in
  // one of 64; D = 64: 8.6 and 8.4)
  const CacheAttnParams &p = tp.a;
  int rows = p.R <= 16 ? 16 : p.R <= 32 ? 32 : 64;
  if (p.T <= 32) rows = short_block(p, D * 2, how.sms, rows, 16);
  if (rows == 16) return launch_t<T, D, 1>(maps, tp, how, s);
  if (rows == 32) return launch_t<T, D, 2>(maps, tp, how, s);
  return launch_t<T, D, 4>(maps, tp, how, s);
}

}  // namespace

bool cache_attn_maps(const CacheAttnParams &p, mgqa_dtype dt, int D, int tile, CUtensorMap (&maps)[4], int &box_rows) {
  const int cols = dt == MGQA_FP32 ? 32 : 64;  // 128 bytes
  const int n0 = p.table ? p.num_pages : p.B, n2 = p.table ? p.page_size : p.cap;
  if ((p.table && p.page_size % 8) || !plain_strides(p.ks, n0, p.Hkv, n2) || !plain_strides(p.vs, n0, p.Hkv, n2) ||
      (p.tree && (!plain_strides(p.kns, p.B, p.Hkv, p.T) || !plain_strides(p.vns, p.B, p.Hkv, p.T)))) {
    box_rows = 0;
    std::memset(maps, 0, sizeof(maps));
    return true;
  }
  box_rows = tile;
  if (p.table)
    for (; p.page_size % box_rows; box_rows /= 2) {}
  const int pages = p.table ? p.num_pages : p.B, slots = p.table ? p.page_size : p.cap;
  if (!make_tma_map_4d(&maps[0], dt, p.k, pages, p.Hkv, slots, D, p.ks, cols, box_rows, true) ||
      !make_tma_map_4d(&maps[1], dt, p.v, pages, p.Hkv, slots, D, p.vs, cols, box_rows, true))
    return false;
  maps[2] = maps[0];
  maps[3] = maps[1];
  return !p.tree || (make_tma_map_4d(&maps[2], dt, p.kn, p.B, p.Hkv, p.T, D, p.kns, cols, tile, true) &&
                     make_tma_map_4d(&maps[3], dt, p.vn, p.B, p.Hkv, p.T, D, p.vns, cols, tile, true));
}

// Up to 32 rows; up to 64 for short calls, where a cluster saves a launch: on
// longer ones the tensor-memory kernel is ahead (64 rows, 4 requests of up to
// 131072: 305 us here, 234 us there). One request, full: 2 KV heads, D = 64, 4096
// slots 11.2 us here, 12.9 there; 8 KV heads, D = 128, 256 slots 11.2 and 13.1, but
// 1024 slots 18.0 and 12.8 and 4096 23.7 and 17.0 (eight units leave no SMs for
// smaller blocks), which a rule on the reads alone misses. And what that kernel
// does not take.
bool cache_attn_tma_takes(const CacheAttnParams &p, mgqa_dtype dt, int D) {
  return p.R <= 32 || (p.R <= 64 && short_call(p, D * 2)) || !cache_attn_tc_takes(p);
}

mgqa_status launch_cache_attn_tma(const CacheAttnParams &p, mgqa_dtype dt, int D, const CacheAttnLaunch &how,
                                  cudaStream_t s) {
  TmaParams tp{};
  tp.a = p;
  CUtensorMap maps[4];
  if (!cache_attn_maps(p, dt, D, kTile, maps, tp.box_rows))
    return fail(MGQA_ERR_CUDA, "cuTensorMapEncodeTiled failed for the cache");
  if (dt == MGQA_BF16)
    return D == 64 ? launch_d<__nv_bfloat16, 64>(maps, tp, how, s) : launch_d<__nv_bfloat16, 128>(maps, tp, how, s);
  return D == 64 ? launch_d<__half, 64>(maps, tp, how, s) : launch_d<__half, 128>(maps, tp, how, s);
}

}  // namespace mgqa
