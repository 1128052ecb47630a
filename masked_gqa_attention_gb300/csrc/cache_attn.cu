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
// R = 64 the reads are the floor. K and V rows arrive by 16-byte asynchronous
// copies, one page lookup per row and no rule on the page size, into a ring of
// tiles; rows are stored with their 16-byte pieces exchanged (piece ^ row % 8),
// which makes every matrix load conflict-free.
//   16-bit: the products on mma.sync (m16n8k16). A CTA holds 16, 32 or 64 rows;
//     with 16 or 32 rows its four warps split each tile's keys, so a single
//     token's few rows still use the whole CTA, and join once at the end.
//   fp32: the CUDA cores, register tiles of 1 x 4 or 4 x 4 scores per thread.
#include <algorithm>
#include <cmath>

#include "cache_sched.cuh"

namespace mgqa {
namespace {

constexpr int kThreads = 128;  // 16-bit kernel
constexpr int kSimtThreads = 256;

// 16 bytes global -> shared, or 16 zero bytes (nothing is read then).
MGQA_DEV void cp_async16_or_zero(uint32_t dst, const void *src, bool take) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src),
               "r"(take ? 16 : 0)
               : "memory");
}

// The rows of one tile, fetched by a whole CTA. One thread a row finds where it
// lies (the page two tiles ahead of its use, so the table is never waited for)
// and leaves the two offsets in shared memory; then pass u of thread tid brings
// 16-byte piece tid % CH of row tid / CH + u * RPP. (Every thread finding its own
// rows' addresses took three times the instructions of the copies themselves.)
constexpr int64_t kHidden = -1, kMissing = -2;  // offsets of rows that nobody sees, of a page that is not there
struct RowOffsets {
  longlong2 at[2][kTile];  // of alternating tiles: bytes of the row in K and in V
};

template <typename T, int D, int THREADS>
struct TileLoader {
  static constexpr int CH = D * (int)sizeof(T) / 16;
  static constexpr int RPP = THREADS / CH;
  static constexpr int NP = kTile / RPP;
  static_assert(THREADS % CH == 0 && kTile % RPP == 0 && THREADS >= kTile, "whole rows per pass");
  int page;  // of this thread's row of the tile that is placed next (-2: hidden, -1: missing)

  MGQA_DEV void look_up(const CacheAttnParams &p, const RowPlan &rp, int b, int i, int tid) {
    if (tid >= kTile) return;
    int kind;
    const int j = first_key(rp, i, 6, kind) + tid;
    page = wanted(rp, kind, j) ? (kind ? b : page_of(p, b, j)) : -2;
  }
  // Row offsets of tile i, whose page was looked up, to `off`.
  MGQA_DEV void place(const CacheAttnParams &p, const RowPlan &rp, int g, int i, int tid, longlong2 *off) const {
    if (tid >= kTile) return;
    int kind;
    const int j = first_key(rp, i, 6, kind) + tid;
    const int64_t *ks = kind ? p.kns : p.ks, *vs = kind ? p.vns : p.vs;
    const int s = kind ? j : slot_in_page(p, j);
    longlong2 at = make_longlong2(page == -2 ? kHidden : kMissing, 0);
    if (page >= 0)
      at = make_longlong2(((int64_t)page * ks[0] + (int64_t)g * ks[1] + (int64_t)s * ks[2]) * (int64_t)sizeof(T),
                          ((int64_t)page * vs[0] + (int64_t)g * vs[1] + (int64_t)s * vs[2]) * (int64_t)sizeof(T));
    off[tid] = at;
  }
  // Issues tile i into kdst / vdst (shared addresses; row_addr(r, piece)); ok[r]
  // tells whether row r counts, *bad is raised when a page is missing.
  template <typename RowAddr>
  MGQA_DEV void issue(const CacheAttnParams &p, const RowPlan &rp, int i, int tid, const longlong2 *off,
                      uint32_t kdst, uint32_t vdst, uint8_t *ok, int *bad, RowAddr row_addr) const {
    const bool kind = i >= rp.np;
    const int piece = tid % CH;
    const char *kb = static_cast<const char *>(kind ? p.kn : p.k) + piece * 16;
    const char *vb = static_cast<const char *>(kind ? p.vn : p.v) + piece * 16;
#pragma unroll
    for (int u = 0; u < NP; ++u) {
      const int r = tid / CH + u * RPP;
      const longlong2 at = off[r];
      const bool take = at.x >= 0;
      // a row that does not count gives zeros and is not read (any valid address)
      cp_async16_or_zero(kdst + row_addr(r, piece), take ? kb + at.x : static_cast<const char *>(p.k), take);
      cp_async16_or_zero(vdst + row_addr(r, piece), take ? vb + at.y : static_cast<const char *>(p.v), take);
      if (piece == 0) {
        ok[r] = take;
        if (at.x == kMissing) {
          *bad = 1;
          report_error(p.err, MGQA_ERR_INVALID_ARG);
        }
      }
    }
  }
};

// ---- 16-bit: mma.sync -----------------------------------------------------------

template <int D, int WM>
struct MmaCfg {
  static constexpr int WK = 4 / WM;        // warps that share a tile's keys
  static constexpr int ROWS = 16 * WM;     // query rows of a CTA
  static constexpr int KW = kTile / WK;    // keys of a warp in a tile
  static constexpr int STAGES = D == 128 ? 3 : 4;
  static constexpr int TILEB = kTile * D * 2;  // bytes of a K (or V) tile
  static constexpr int OP = D + 4;             // row pitch of the joined output (floats)
  static constexpr int ring = STAGES * 2 * TILEB;
  static_assert(WK * ROWS * OP * 4 <= ring, "the joined output fits in the ring");
  struct Misc {
    Drafts<kMaxDrafts> drafts;
    LocateScratch<kThreads> scratch;
    float wm[WK][ROWS], wl[WK][ROWS];
    RowOffsets off;
    uint8_t ok[STAGES][kTile];
    int bad, maxdepth;
  };
  static constexpr int smem = ring + (int)sizeof(Misc) + 128;
  // byte of piece c of row r in a tile
  static MGQA_DEV uint32_t at(int r, int c) { return (uint32_t)(r * (D * 2) + ((c ^ (r & 7)) << 4)); }
};

template <typename T, int D, int WM>
__global__ void __launch_bounds__(kThreads, 2)
cache_attn_kernel(const __grid_constant__ CacheAttnParams p) {
  using Cfg = MmaCfg<D, WM>;
  constexpr int WK = Cfg::WK, ROWS = Cfg::ROWS, KW = Cfg::KW, STAGES = Cfg::STAGES;
  extern __shared__ __align__(128) unsigned char smem_raw[];
  unsigned char *ring = smem_raw;
  auto &sm = *reinterpret_cast<typename Cfg::Misc *>(smem_raw + Cfg::ring);
  const uint32_t ring_a = smem_u32(ring);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int wm = warp / WK, wk = warp % WK;
  const int gq = lane >> 2, tq = lane & 3, mi = lane >> 3, rr = lane & 7;

  grid_dependency_wait();
  allow_dependents();  // the merge kernel; lengths and tables are final from here on
  const Located loc = locate<kThreads>(p, sm.scratch, gridDim.x, blockIdx.x, blockIdx.x == 0);
  Walker walk;
  walk.start(p, loc, blockIdx.x);
  Piece pc;
  if (tid == 0) tell_cut(p, blockIdx.x, nullptr);
  int staged = -1;  // request whose drafts are staged

  while (walk.next(p, pc)) {
    if (tid == 0) tell_cut(p, blockIdx.x, &pc);
    const RowPlan &rp = pc.rp;
    const int b = pc.b, g = pc.g, t0 = pc.t0, t1 = pc.t1;
    const PieceOut po = out_of(p, pc, blockIdx.x);
    const int row0 = po.row0;

    // ---- the first tiles' copies, then q and the drafts' masks
    TileLoader<T, D, kThreads> ld;
    const int nt = t1 - t0;
    if (tid == 0) {
      sm.bad = 0;
      if (staged != b) sm.maxdepth = 0;
    }
    __syncthreads();  // (also: the previous piece's readers are done with the ring)
    auto issue = [&](int i) {
      if (i < nt) {
        const int st = i % STAGES;
        ld.issue(p, rp, t0 + i, tid, sm.off.at[i & 1], ring_a + st * 2 * Cfg::TILEB,
                 ring_a + st * 2 * Cfg::TILEB + Cfg::TILEB, sm.ok[st], &sm.bad, Cfg::at);
      }
      cp_async_commit();
    };
    auto look_up = [&](int i) {
      if (i < nt) ld.look_up(p, rp, b, t0 + i, tid);
    };
    auto place = [&](int i) {  // (a barrier before tile i is issued, and one since tile i - 2 was)
      if (i < nt) ld.place(p, rp, g, t0 + i, tid, sm.off.at[i & 1]);
    };
    look_up(0);
#pragma unroll
    for (int i = 0; i < STAGES - 1; ++i) {
      place(i);
      look_up(i + 1);
      __syncthreads();
      issue(i);
    }
    place(STAGES - 1);
    look_up(STAGES);

    uint32_t qa[D / 16][4];
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      const int row = row0 + wm * 16 + gq + 8 * half;
      const bool in = row < p.R;
      const int t = in ? row / p.n_rep : 0, h = g * p.n_rep + (in ? row % p.n_rep : 0);
      const T *src = static_cast<const T *>(p.q) + (int64_t)b * p.qs[0] + (int64_t)h * p.qs[1] + (int64_t)t * p.qs[2];
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk) {
        qa[kk][half] = in ? *reinterpret_cast<const uint32_t *>(src + kk * 16 + 2 * tq) : 0u;
        qa[kk][2 + half] = in ? *reinterpret_cast<const uint32_t *>(src + kk * 16 + 8 + 2 * tq) : 0u;
      }
    }
    const bool need_drafts = p.tree && (p.window != kNoWindow || t1 > rp.np);
    if (need_drafts && staged != b) {
      stage_drafts(p, sm.drafts, b, rp.live, tid, kThreads);
      __syncthreads();
      int md = 0;
      for (int t = tid; t < rp.live; t += kThreads) md = max(md, sm.drafts.depth[t]);
      if (md) atomicMax(&sm.maxdepth, md);
      __syncthreads();
      staged = b;
    }
    RowSight sight[2];
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      const int row = row0 + wm * 16 + gq + 8 * half;
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

    for (int i = 0; i < nt; ++i) {
      cp_async_wait<STAGES - 2>();
      __syncthreads();  // tile i landed for everyone, and tile i - 1 has been read
      issue(i + STAGES - 1);
      place(i + STAGES);
      look_up(i + STAGES + 1);
      const int st = i % STAGES;
      const unsigned char *kt = ring + st * 2 * Cfg::TILEB, *vt = kt + Cfg::TILEB;
      const int key0 = wk * KW;  // this warp's keys of the tile
      float s[KW / 8][4];
#pragma unroll
      for (int nn = 0; nn < KW / 8; ++nn) s[nn][0] = s[nn][1] = s[nn][2] = s[nn][3] = 0.f;
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk)
#pragma unroll
        for (int np = 0; np < KW / 16; ++np) {
          uint32_t b0, b1, b2, b3;
          ldmatrix_x4(b0, b1, b2, b3, kt + Cfg::at(key0 + np * 16 + (mi >> 1) * 8 + rr, 2 * kk + (mi & 1)));
          mma_16816<T>(s[2 * np], qa[kk][0], qa[kk][1], qa[kk][2], qa[kk][3], b0, b1);
          mma_16816<T>(s[2 * np + 1], qa[kk][0], qa[kk][1], qa[kk][2], qa[kk][3], b2, b3);
        }
      // scale and mask
      int kind;
      const int k0 = first_key(rp, t0 + i, 6, kind);
      const bool full = !kind && !sm.bad && k0 + kTile <= rp.n &&
                        (k0 >= lo_all || k0 + kTile <= min(p.sinks, rp.s_end));
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
            const bool see = sm.ok[st][c] && (kind ? sees_draft(p, sm.drafts, rs, rp.n, k0 + c)
                                                   : sees_cached(p, rs, k0 + c));
            s[nn][e] = see ? s[nn][e] * p.scale_log2 : -INFINITY;
          }
      }
      float mx[2] = {m[0], m[1]};
#pragma unroll
      for (int nn = 0; nn < KW / 8; ++nn) {
        mx[0] = fmaxf(mx[0], fmaxf(s[nn][0], s[nn][1]));
        mx[1] = fmaxf(mx[1], fmaxf(s[nn][2], s[nn][3]));
      }
      float mb[2];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        mx[e] = fmaxf(mx[e], __shfl_xor_sync(0xffffffffu, mx[e], 1));
        mx[e] = fmaxf(mx[e], __shfl_xor_sync(0xffffffffu, mx[e], 2));
        mb[e] = mx[e] == -INFINITY ? 0.f : mx[e];  // nothing seen yet: every weight is 0
      }
      if (__any_sync(0xffffffffu, mx[0] != m[0] || mx[1] != m[1])) {
        const float f0 = fast_exp2(m[0] - mb[0]), f1s = fast_exp2(m[1] - mb[1]);
        l[0] *= f0;
        l[1] *= f1s;
#pragma unroll
        for (int d = 0; d < D / 8; ++d) {
          o[d][0] *= f0;
          o[d][1] *= f0;
          o[d][2] *= f1s;
          o[d][3] *= f1s;
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
#pragma unroll
      for (int kp = 0; kp < KW / 16; ++kp) {
        const uint32_t a0 = pack2<T>(s[2 * kp][0], s[2 * kp][1]), a1 = pack2<T>(s[2 * kp][2], s[2 * kp][3]);
        const uint32_t a2 = pack2<T>(s[2 * kp + 1][0], s[2 * kp + 1][1]);
        const uint32_t a3 = pack2<T>(s[2 * kp + 1][2], s[2 * kp + 1][3]);
#pragma unroll
        for (int dp = 0; dp < D / 16; ++dp) {
          uint32_t b0, b1, b2, b3;
          ldmatrix_x4_trans(b0, b1, b2, b3, vt + Cfg::at(key0 + kp * 16 + (mi & 1) * 8 + rr, 2 * dp + (mi >> 1)));
          mma_16816<T>(o[2 * dp], a0, a1, a2, a3, b0, b1);
          mma_16816<T>(o[2 * dp + 1], a0, a1, a2, a3, b2, b3);
        }
      }
    }
    cp_async_wait<0>();
    // ---- join the warps that shared the keys, through the ring
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      l[e] += __shfl_xor_sync(0xffffffffu, l[e], 1);
      l[e] += __shfl_xor_sync(0xffffffffu, l[e], 2);
      if (!sight[e].ok) {  // scores of a row that sees nothing were never masked in full tiles
        m[e] = -INFINITY;
        l[e] = 0.f;
      }
      if (tq == 0) {
        sm.wm[wk][wm * 16 + gq + 8 * e] = m[e];
        sm.wl[wk][wm * 16 + gq + 8 * e] = l[e];
      }
    }
    __syncthreads();  // every warp is done with the ring
    float *jo = reinterpret_cast<float *>(ring);
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int r = wm * 16 + gq + 8 * e;
      float mr = -INFINITY;
#pragma unroll
      for (int w = 0; w < WK; ++w) mr = fmaxf(mr, sm.wm[w][r]);
      const float fr = m[e] == -INFINITY ? 0.f : fast_exp2(m[e] - mr);
#pragma unroll
      for (int d = 0; d < D / 8; ++d)
        *reinterpret_cast<float2 *>(jo + (wk * ROWS + r) * Cfg::OP + d * 8 + 2 * tq) =
            fr == 0.f ? make_float2(0.f, 0.f) : make_float2(o[d][2 * e] * fr, o[d][2 * e + 1] * fr);
    }
    __syncthreads();
    for (int u = tid; u < po.rows * (D / 4); u += kThreads) {
      const int r = u / (D / 4), d = (u % (D / 4)) * 4;
      float mr = -INFINITY, lr = 0.f;
      float acc[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int w = 0; w < WK; ++w) mr = fmaxf(mr, sm.wm[w][r]);
#pragma unroll
      for (int w = 0; w < WK; ++w) {
        if (sm.wm[w][r] == -INFINITY) continue;
        lr = fmaf(sm.wl[w][r], fast_exp2(sm.wm[w][r] - mr), lr);
        const float4 x = *reinterpret_cast<const float4 *>(jo + (w * ROWS + r) * Cfg::OP + d);
        acc[0] += x.x;
        acc[1] += x.y;
        acc[2] += x.z;
        acc[3] += x.w;
      }
      RowOut<T, D, ROWS>(p, po, r, mr, lr, d == 0).put(d, acc);
    }
  }
}

// ---- fp32: CUDA cores -------------------------------------------------------------

template <int D, int RPT>
struct SimtCfg {
  static constexpr int ROWS = 16 * RPT;  // thread (ty, tx): rows ty + 16 i, keys tx + 16 j
  static constexpr int RP = D + 4;       // row pitch of q, K and V (floats): conflict-free 16-byte reads
  static constexpr int PP = kTile + 4;   // row pitch of the weights
  static constexpr int STAGES = 2;
  static constexpr int TILEF = kTile * RP;
  static constexpr int floats = STAGES * 2 * TILEF + ROWS * RP + ROWS * PP;
  struct Misc {
    Drafts<kMaxDrafts> drafts;
    LocateScratch<kSimtThreads> scratch;
    RowOffsets off;
    uint8_t ok[STAGES][kTile];
    int bad, maxdepth;
  };
  static constexpr int smem = floats * 4 + (int)sizeof(Misc) + 128;
  static MGQA_DEV uint32_t at(int r, int c) { return (uint32_t)(r * (RP * 4) + c * 16); }
};

template <int D, int RPT>
__global__ void __launch_bounds__(kSimtThreads, 1)
cache_attn_fp32_kernel(const __grid_constant__ CacheAttnParams p) {
  using Cfg = SimtCfg<D, RPT>;
  constexpr int ROWS = Cfg::ROWS, RP = Cfg::RP, PP = Cfg::PP, STAGES = Cfg::STAGES;
  extern __shared__ __align__(128) unsigned char smem_raw[];
  float *ring = reinterpret_cast<float *>(smem_raw);
  float *qs = ring + STAGES * 2 * Cfg::TILEF, *ps = qs + ROWS * RP;
  auto &sm = *reinterpret_cast<typename Cfg::Misc *>(smem_raw + Cfg::floats * 4);
  const uint32_t ring_a = smem_u32(ring);
  const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;

  grid_dependency_wait();
  allow_dependents();
  const Located loc = locate<kSimtThreads>(p, sm.scratch, gridDim.x, blockIdx.x, blockIdx.x == 0);
  Walker walk;
  walk.start(p, loc, blockIdx.x);
  Piece pc;
  if (tid == 0) tell_cut(p, blockIdx.x, nullptr);
  int staged = -1;

  while (walk.next(p, pc)) {
    if (tid == 0) tell_cut(p, blockIdx.x, &pc);
    const RowPlan &rp = pc.rp;
    const int b = pc.b, g = pc.g, t0 = pc.t0, t1 = pc.t1;
    const PieceOut po = out_of(p, pc, blockIdx.x);
    const int row0 = po.row0;
    TileLoader<float, D, kSimtThreads> ld;
    const int nt = t1 - t0;
    if (tid == 0) {
      sm.bad = 0;
      if (staged != b) sm.maxdepth = 0;
    }
    __syncthreads();
    auto issue = [&](int i) {
      if (i < nt) {
        const int st = i % STAGES;
        ld.issue(p, rp, t0 + i, tid, sm.off.at[i & 1], ring_a + st * 2 * Cfg::TILEF * 4,
                 ring_a + (st * 2 + 1) * Cfg::TILEF * 4, sm.ok[st], &sm.bad, Cfg::at);
      }
      cp_async_commit();
    };
    auto look_up = [&](int i) {
      if (i < nt) ld.look_up(p, rp, b, t0 + i, tid);
    };
    auto place = [&](int i) {  // (a barrier before tile i is issued, and one since tile i - 2 was)
      if (i < nt) ld.place(p, rp, g, t0 + i, tid, sm.off.at[i & 1]);
    };
    look_up(0);
    place(0);
    look_up(1);
    __syncthreads();
    issue(0);
    place(1);
    look_up(2);
    __syncthreads();
    for (int u = tid; u < ROWS * (D / 4); u += kSimtThreads) {  // q, in log2 units
      const int r = u / (D / 4), d = (u % (D / 4)) * 4, row = row0 + r;
      float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
      if (row < p.R)
        x = *reinterpret_cast<const float4 *>(static_cast<const float *>(p.q) + (int64_t)b * p.qs[0] +
                                              (int64_t)(g * p.n_rep + row % p.n_rep) * p.qs[1] +
                                              (int64_t)(row / p.n_rep) * p.qs[2] + d);
      *reinterpret_cast<float4 *>(qs + r * RP + d) = x;
    }
    const bool need_drafts = p.tree && (p.window != kNoWindow || t1 > rp.np);
    if (need_drafts && staged != b) {
      stage_drafts(p, sm.drafts, b, rp.live, tid, kSimtThreads);
      __syncthreads();
      int md = 0;
      for (int t = tid; t < rp.live; t += kSimtThreads) md = max(md, sm.drafts.depth[t]);
      if (md) atomicMax(&sm.maxdepth, md);
      __syncthreads();
      staged = b;
    }
    RowSight sight[RPT];
#pragma unroll
    for (int i = 0; i < RPT; ++i) {
      const int row = row0 + ty + 16 * i;
      sight[i].t = row / p.n_rep;
      sight[i].ok = row < p.R && (!p.tree || sight[i].t < rp.live);
      const int pt = p.tree ? rp.n + (need_drafts && sight[i].ok ? sm.drafts.depth[sight[i].t] : 0) : rp.n - 1;
      sight[i].lo = pt - p.window + 1;
    }
    const int lo_all = rp.n + (p.tree ? (need_drafts ? sm.maxdepth : 0) : -1) - p.window + 1;

    constexpr int ND = D / 64;  // float4 columns of a thread: tx * 4 + 64 c
    float o[RPT][ND][4], m[RPT], l[RPT];
#pragma unroll
    for (int i = 0; i < RPT; ++i) {
      m[i] = -INFINITY;
      l[i] = 0.f;
#pragma unroll
      for (int c = 0; c < ND; ++c) o[i][c][0] = o[i][c][1] = o[i][c][2] = o[i][c][3] = 0.f;
    }
    for (int i = 0; i < nt; ++i) {
      issue(i + 1);  // its buffer's readers passed the barrier that ends a tile
      place(i + 2);
      look_up(i + 3);
      cp_async_wait<1>();
      __syncthreads();
      const int st = i % STAGES;
      const float *kt = ring + st * 2 * Cfg::TILEF, *vt = kt + Cfg::TILEF;
      float s[RPT][4];
#pragma unroll
      for (int a = 0; a < RPT; ++a) s[a][0] = s[a][1] = s[a][2] = s[a][3] = 0.f;
#pragma unroll 4
      for (int d = 0; d < D; d += 4) {
        float4 kv[4];
#pragma unroll
        for (int c = 0; c < 4; ++c) kv[c] = *reinterpret_cast<const float4 *>(kt + (tx + 16 * c) * RP + d);
#pragma unroll
        for (int a = 0; a < RPT; ++a) {
          const float4 qv = *reinterpret_cast<const float4 *>(qs + (ty + 16 * a) * RP + d);
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            s[a][c] = fmaf(qv.x, kv[c].x, s[a][c]);
            s[a][c] = fmaf(qv.y, kv[c].y, s[a][c]);
            s[a][c] = fmaf(qv.z, kv[c].z, s[a][c]);
            s[a][c] = fmaf(qv.w, kv[c].w, s[a][c]);
          }
        }
      }
      int kind;
      const int k0 = first_key(rp, t0 + i, 6, kind);
      const bool full = !kind && !sm.bad && k0 + kTile <= rp.n &&
                        (k0 >= lo_all || k0 + kTile <= min(p.sinks, rp.s_end));
#pragma unroll
      for (int a = 0; a < RPT; ++a) {
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const int col = tx + 16 * c;
          const bool see = full || (sm.ok[st][col] && (kind ? sees_draft(p, sm.drafts, sight[a], rp.n, k0 + col)
                                                            : sees_cached(p, sight[a], k0 + col)));
          s[a][c] = see ? s[a][c] * p.scale_log2 : -INFINITY;
        }
        float mx = fmaxf(m[a], fmaxf(fmaxf(s[a][0], s[a][1]), fmaxf(s[a][2], s[a][3])));
#pragma unroll
        for (int off = 1; off < 16; off <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, off));
        const float mb = mx == -INFINITY ? 0.f : mx;
        const float fa = exp2f(m[a] - mb);
        m[a] = mx;
        l[a] *= fa;
#pragma unroll
        for (int c = 0; c < ND; ++c)
#pragma unroll
          for (int e = 0; e < 4; ++e) o[a][c][e] *= fa;
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const float w = exp2f(s[a][c] - mb);
          l[a] += w;
          ps[(ty + 16 * a) * PP + tx + 16 * c] = w;
        }
      }
      __syncwarp();  // a row's weights come from the 16 lanes that read them
#pragma unroll 2
      for (int k = 0; k < kTile; k += 4) {
        float4 w[RPT];
#pragma unroll
        for (int a = 0; a < RPT; ++a) w[a] = *reinterpret_cast<const float4 *>(ps + (ty + 16 * a) * PP + k);
#pragma unroll
        for (int kk = 0; kk < 4; ++kk)
#pragma unroll
          for (int c = 0; c < ND; ++c) {
            const float4 vv = *reinterpret_cast<const float4 *>(vt + (k + kk) * RP + tx * 4 + 64 * c);
#pragma unroll
            for (int a = 0; a < RPT; ++a) {
              const float wa = kk == 0 ? w[a].x : kk == 1 ? w[a].y : kk == 2 ? w[a].z : w[a].w;
              o[a][c][0] = fmaf(wa, vv.x, o[a][c][0]);
              o[a][c][1] = fmaf(wa, vv.y, o[a][c][1]);
              o[a][c][2] = fmaf(wa, vv.z, o[a][c][2]);
              o[a][c][3] = fmaf(wa, vv.w, o[a][c][3]);
            }
          }
      }
      __syncthreads();
    }
    cp_async_wait<0>();
#pragma unroll
    for (int a = 0; a < RPT; ++a) {
      float ls = l[a];
#pragma unroll
      for (int off = 1; off < 16; off <<= 1) ls += __shfl_xor_sync(0xffffffffu, ls, off);
      const int r = ty + 16 * a;
      const bool none = !sight[a].ok;
      if (r < po.rows) {
        const RowOut<float, D, ROWS> dst(p, po, r, none ? -INFINITY : m[a], none ? 0.f : ls, tx == 0);
#pragma unroll
        for (int c = 0; c < ND; ++c) {
          if (none) o[a][c][0] = o[a][c][1] = o[a][c][2] = o[a][c][3] = 0.f;
          dst.put(tx * 4 + 64 * c, o[a][c]);
        }
      }
    }
  }
}

// ---- joining the partial results -------------------------------------------------

constexpr int kMergeThreads = 128;

// Block (unit or run, 16 rows, 32 features): joins the pieces of the unit, if it
// was cut, in the order of the runs. A thread has four features of a
// row; partial results are read in runs of 16 rows x 16 bytes.
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
  switch (block_rows) {
    case 4: return launch_merge<T, D, 4>(p, grid, s);
    case 8: return launch_merge<T, D, 8>(p, grid, s);
    case 16: return launch_merge<T, D, 16>(p, grid, s);
    case 32: return launch_merge<T, D, 32>(p, grid, s);
    case 64: return launch_merge<T, D, 64>(p, grid, s);
    case 128: return launch_merge<T, D, 128>(p, grid, s);
    case 256: return launch_merge<T, D, 256>(p, grid, s);
    default: return fail(MGQA_ERR_UNSUPPORTED, "merge: blocks of %d rows", block_rows);
  }
}

template <typename T, int D, int BR, typename Kern>
mgqa_status launch_with(Kern kern, int smem, std::atomic<uint64_t> &attr, int threads, int per_sm, CacheAttnParams p,
                        const CacheAttnLaunch &how, cudaStream_t s) {
  mgqa_status st = ensure_smem_attr(kern, smem, attr, "cache attention kernel");
  if (st != MGQA_OK) return st;
  p.block_rows = BR;
  p.RB = (p.R + BR - 1) / BR;
  p.tile_shift = 6;
  p.lead = 2;
  p.min_run = 4;
  const int64_t tiles = (int64_t)p.B * p.Hkv * p.RB * (most_tiles(p) + p.lead);
  const int grid = (int)std::max<int64_t>(1, std::min<int64_t>(std::min(how.sms * per_sm, kCacheAttnMaxCtas), tiles));
  set_partials(p, how.workspace, grid, BR, D);
  const cudaError_t e = launch_pdl(kern, dim3(grid), dim3(threads), smem, s, p);
  if (e != cudaSuccess) return fail(MGQA_ERR_CUDA, "cache attention launch: %s", cudaGetErrorString(e));
  return launch_merge<T, D, BR>(p, grid, s);
}

template <typename T, int D, int WM>
mgqa_status launch_mma(const CacheAttnParams &p, const CacheAttnLaunch &how, cudaStream_t s) {
  static std::atomic<uint64_t> attr{0};
  using Cfg = MmaCfg<D, WM>;
  return launch_with<T, D, Cfg::ROWS>(cache_attn_kernel<T, D, WM>, Cfg::smem, attr, kThreads, 2, p, how, s);
}

template <typename T, int D>
mgqa_status launch_16bit(const CacheAttnParams &p, const CacheAttnLaunch &how, cudaStream_t s) {
  // the smallest row block that holds the unit's rows
  if (p.R <= 16) return launch_mma<T, D, 1>(p, how, s);
  if (p.R <= 32) return launch_mma<T, D, 2>(p, how, s);
  return launch_mma<T, D, 4>(p, how, s);
}

template <int D, int RPT>
mgqa_status launch_simt(const CacheAttnParams &p, const CacheAttnLaunch &how, cudaStream_t s) {
  static std::atomic<uint64_t> attr{0};
  using Cfg = SimtCfg<D, RPT>;
  return launch_with<float, D, Cfg::ROWS>(cache_attn_fp32_kernel<D, RPT>, Cfg::smem, attr, kSimtThreads, 1, p, how, s);
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
  if (cache_attn_f32_takes(p, a.dtype)) return launch_cache_attn_f32(p, a.D, how, s);
  if (cache_attn_tma_takes(p, a.dtype, a.D)) return launch_cache_attn_tma(p, a.dtype, a.D, how, s);
  if (cache_attn_tc_takes(p, a.dtype)) return launch_cache_attn_tc(p, a.dtype, a.D, how, s);
  if (a.dtype == MGQA_BF16)
    return a.D == 64 ? launch_16bit<__nv_bfloat16, 64>(p, how, s)
                     : launch_16bit<__nv_bfloat16, 128>(p, how, s);
  if (a.dtype == MGQA_FP16)
    return a.D == 64 ? launch_16bit<__half, 64>(p, how, s) : launch_16bit<__half, 128>(p, how, s);
  if (a.D == 64)
    return p.R <= 16 ? launch_simt<64, 1>(p, how, s) : launch_simt<64, 4>(p, how, s);
  return p.R <= 16 ? launch_simt<128, 1>(p, how, s) : launch_simt<128, 4>(p, how, s);
}

}  // namespace mgqa
