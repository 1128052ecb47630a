// Attention of the last T cached tokens of every request over a cache in 4 bits
// (cache_q4.cuh has the records and the products).
//
// Query t of request b, with n = kv_len[b], stands at position pos = n - T + t
// (below 0: it sees nothing) and sees slot j when
//   j <= pos and (no window, or pos - j < window, or j < sinks).
//
// Every visible record is read once per KV head and block of query rows; a warp
// spends some 900 instructions on 64 keys of 128 features, which the reads take
// 435 cycles for, so the kernel has to keep both going. Each warp streams tiles of
// 32 keys of its own through a ring in shared memory: one bulk copy per page and
// tensor, counted on the warp's own barrier, and no barrier between warps inside a
// unit. Rows of queries are the first operand of the scores and the second one of
// the outputs (transposed), so the scores' accumulators are the weights' operand as
// they are.
//
// Weights: p is 2^14 at most (the maximum is subtracted 14 short), and p times a
// scale is divided by the largest scale's power of two so far, so the fp16 operand
// keeps 2^-11 of it down to 2^-28 of the largest (2^-22 in two terms for fp32
// calls). Sums of weights and outputs are fp32, a tile's from the tensor cores and
// those of the tiles in rounded additions: codes and least values are sums of one
// sign that nearly cancel, and the tensor cores' accumulators truncate (32 rows of
// 98000 keys: 0.0066 of the outputs' size from 64 bits with running accumulators).
// For the same reason fp16 and fp32 calls take the codes from their middle,
//   out_d = sum_j (p_j scale_jg) (u_jd - 8) + sum_j p_j (least_jg + 8 scale_jg),
// so that roundings of the weights are not multiplied by terms that cancel (the -8
// by products with a constant; fp16: 0.0005 of the outputs' size without, where the
// outputs' own rounding makes 0.0002). In bf16 the outputs' rounding hides it.
//
// The work is cut as for the other cache attention (cache_sched.cuh): equal runs of
// tiles and the merge kernel for long calls, a cluster per unit for short ones.
#include <algorithm>
#include <cmath>

#include "cache_producer.cuh"
#include "cache_q4.cuh"

namespace mgqa {
namespace {

constexpr int kWarps = 4;
constexpr int kThreads = 32 * kWarps;
constexpr int kShift = 5, kKeys = 32;  // keys of a tile
constexpr int kMostCtas = 512;         // partial results: two per CTA

struct Q4Params {
  TmaParams t;  // (its strides of k and v are bytes)
  int32_t run_slots;  // slots of a page that lie one after the other: page_size (or cap), or 1
};

template <int D, int RT>
struct Cfg {
  static constexpr int ROWS = 8 * RT;
  static constexpr int STAGES = RT == 4 ? 4 : 3;
  static constexpr int CTAS = 2;  // of an SM
  static constexpr int TILEB = kKeys * Q4<D>::REC;
  static constexpr int ring = kWarps * STAGES * 2 * TILEB;
  static constexpr int OP = D + 4;  // row pitch of a CTA's result (floats)
  struct Misc {
    float res[ROWS * OP];             // the CTA's result, 16-byte aligned
    float wm[kWarps][ROWS], wl[kWarps][ROWS];
    float2 ml[ROWS];
    LocateScratch<kThreads> scratch;
    uint64_t full[kWarps][STAGES];
    uint32_t ok[kWarps][STAGES];      // which keys of a stage's tile count
  };
  static constexpr int smem = ring + (int)sizeof(Misc);
};

// The tiles of a warp, in order, ahead of their use: every kWarps-th of each piece.
struct Feed {
  Pieces pieces;
  Piece pc;
  int t, page;
  bool live;

  MGQA_DEV void settle(const Q4Params &p, int warp) {  // to the next tile that there is
    while (live && t >= pc.t1) {
      live = pieces.next(p.t.a, pc);
      t = pc.t0 + warp;
    }
    if (live) look_up(p);
  }
  MGQA_DEV void start(const Q4Params &p, const Pieces &all, int warp) {
    pieces = all;
    live = true;
    t = 0;
    pc.t1 = 0;
    settle(p, warp);
  }
  // Slots [a, e) of this lane's part of tile t: a page's, or one.
  MGQA_DEV void part(const Q4Params &p, int &k0, int &a, int &e) const {
    const CacheAttnParams &c = p.t.a;
    const int lane = threadIdx.x & 31;
    int kind;
    k0 = first_key(pc.rp, t, kShift, kind);
    const int end = kind ? k0 : min(k0 + kKeys, pc.rp.n);
    if (p.run_slots == 1) {
      a = k0 + lane;
      e = a + 1;
    } else if (c.table) {
      const int i = (c.page_shift >= 0 ? k0 >> c.page_shift : k0 / c.page_size) + lane;
      const int64_t s = (int64_t)i * c.page_size;
      a = (int)min((int64_t)end, max((int64_t)k0, s));
      e = (int)min((int64_t)end, s + c.page_size);
    } else {
      a = lane == 0 ? k0 : end;
      e = end;
    }
    e = min(e, end);
    if (e <= pc.rp.lo && a >= pc.rp.s_end) e = a;  // between the sinks and the window
  }
  MGQA_DEV void look_up(const Q4Params &p) {
    int k0, a, e;
    part(p, k0, a, e);
    page = a < e ? page_of(p.t.a, pc.b, a) : -2;
  }
  // Starts the copies of the tile that was looked up, and looks the next one up.
  template <int D>
  MGQA_DEV void issue(const Q4Params &p, int warp, unsigned char *dst, uint64_t *full, uint32_t *ok) {
    constexpr int REC = Q4<D>::REC;
    const CacheAttnParams &c = p.t.a;
    const int lane = threadIdx.x & 31;
    int k0, a, e;
    part(p, k0, a, e);
    const bool take = page >= 0;
    if (page == -1) report_error(c.err, MGQA_ERR_INVALID_ARG);
    uint32_t bits = 0u;
    int bytes = 0;
    if (take) {
      bytes = (e - a) * REC;
      bits = low_mask(e - k0) & ~low_mask(a - k0) & (~low_mask(pc.rp.lo - k0) | low_mask(pc.rp.s_end - k0));
    }
    bits = __reduce_or_sync(0xffffffffu, bits);
    const int total = __reduce_add_sync(0xffffffffu, bytes);
    if (lane == 0) {
      *ok = bits;
      mbar_arrive_expect_tx(full, (uint32_t)(2 * total));
    }
    __syncwarp();
    if (take) {
      const int64_t slot = slot_in_page(c, a);
      const char *k = static_cast<const char *>(c.k) + page * c.ks[0] + pc.g * c.ks[1] + slot * c.ks[2];
      const char *v = static_cast<const char *>(c.v) + page * c.vs[0] + pc.g * c.vs[1] + slot * c.vs[2];
      bulk_g2s(dst + (a - k0) * REC, k, (uint32_t)bytes, full);
      bulk_g2s(dst + (kKeys + a - k0) * REC, v, (uint32_t)bytes, full);
    }
    t += kWarps;
    settle(p, warp);
  }
};

template <typename T, int D, int RT>
__global__ void __launch_bounds__(kThreads, (Cfg<D, RT>::CTAS))
cache_q4_kernel(const __grid_constant__ Q4Params qp) {
  using C = Cfg<D, RT>;
  using F = Q4<D>;
  constexpr bool SPLIT = sizeof(T) == 4;
  constexpr bool MIDDLE = !__is_same(T, __nv_bfloat16);  // codes count from 8
  constexpr int ROWS = C::ROWS, STAGES = C::STAGES, NC = F::CHUNKS;
  const CacheAttnParams &p = qp.t.a;
  extern __shared__ __align__(1024) unsigned char smem[];
  auto &sm = *reinterpret_cast<typename C::Misc *>(smem + C::ring);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, gq = lane >> 2, tq = lane & 3;
  unsigned char *ring = smem + warp * (STAGES * 2 * C::TILEB);
  uint64_t *full = sm.full[warp];

  if (lane == 0) {
    for (int s = 0; s < STAGES; ++s) mbar_init(full + s, 1);
    fence_mbarrier_init();
  }
  if (warp == 1) touch_params(qp, lane);
  grid_dependency_wait();
  allow_dependents();
  Pieces pieces{};
  pieces.start<kThreads>(qp.t, sm.scratch);  // (its barrier: the mbarriers are initialised)
  const int S = pieces.S;
  const bool teller = tid == 0 && !S;
  if (teller) tell_cut(p, blockIdx.x, nullptr);

  Feed feed;
  feed.start(qp, pieces, warp);
  int put = 0, it = 0, used = 0;  // tiles started, passed, and used
  bool ok = true;
  const auto start_one = [&] {
    feed.template issue<D>(qp, warp, ring + put % STAGES * 2 * C::TILEB, full + put % STAGES, sm.ok[warp] + put % STAGES);
    ++put;
  };
  for (int s = 0; s < STAGES - 1 && feed.live; ++s) start_one();

  if (pieces.idle())
    for (int r = tid; r < ROWS; r += kThreads) sm.ml[r] = make_float2(-INFINITY, 0.f);  // no share of the unit
  Piece pc;
  while (pieces.next(p, pc)) {
    if (teller) tell_cut(p, blockIdx.x, &pc);
    const RowPlan &rp = pc.rp;
    const PieceOut po = out_of(p, pc, blockIdx.x);
    Q4Row<D, SPLIT> q[RT];
    int pos[RT], lo[RT];
#pragma unroll
    for (int r = 0; r < RT; ++r) {
      const int row = po.row0 + 8 * r + gq;
      const bool in = row < p.R;
      const int t = in ? row / p.n_rep : 0, h = pc.g * p.n_rep + (in ? row - t * p.n_rep : 0);
      q[r].load(in ? static_cast<const T *>(p.q) + (int64_t)pc.b * p.qs[0] + (int64_t)h * p.qs[1] + (int64_t)t * p.qs[2]
                   : static_cast<const T *>(nullptr), tq);
      pos[r] = in ? rp.n - p.T + t : -1;
      lo[r] = pos[r] - p.window + 1;
    }
    // every row of the block sees the keys from `far` (and the sinks) to `near`
    const int near = rp.n - p.T + po.row0 / p.n_rep;
    const int far = rp.n - p.T + (po.row0 + po.rows - 1) / p.n_rep - p.window + 1;

    float o[RT][2 * NC][4], vmin[RT][2], m[RT], l[RT];
    int top = -30;  // 2^top: above every scale of V so far
#pragma unroll
    for (int r = 0; r < RT; ++r) {
      m[r] = -INFINITY;
      l[r] = 0.f;
      vmin[r][0] = vmin[r][1] = 0.f;
#pragma unroll
      for (int c = 0; c < 2 * NC; ++c) o[r][c][0] = o[r][c][1] = o[r][c][2] = o[r][c][3] = 0.f;
    }
    for (int t = pc.t0 + warp; t < pc.t1; t += kWarps, ++it) {
      if (ok && feed.live) start_one();
      const int st = it % STAGES;
      if (ok) ok = __all_sync(0xffffffffu, mbar_wait(full + st, (it / STAGES) & 1, p.err));
      if (!ok) continue;
      used = it + 1;
      const unsigned char *kt = ring + st * 2 * C::TILEB;
      unsigned char *vt = ring + (st * 2 + 1) * C::TILEB;
      const uint32_t okw = sm.ok[warp][st];
      float s[RT][4][2];
      q4_scores<D, RT, SPLIT>(q, kt, s);
      int kind;
      const int k0 = first_key(rp, t, kShift, kind);
      const bool clean = okw == 0xffffffffu;
      const bool all = clean && k0 + kKeys - 1 <= near && (k0 >= far || k0 + kKeys <= p.sinks);
      const uint4 vpar = *reinterpret_cast<const uint4 *>(vt + lane * F::REC + F::CODES);
      uint32_t big = 0u;
      if (clean || (okw >> lane & 1u)) {
        big = __vmaxu2(vpar.x, vpar.y);
        big = max(big & 0xffffu, big >> 16);
      } else {  // what lies there may be anything: it counts as 0
        *reinterpret_cast<uint4 *>(vt + lane * F::REC + F::CODES) = make_uint4(0u, 0u, 0u, 0u);
      }
      if (!clean) {
        fence_proxy_async_smem();  // (the next copy to this place comes after these stores)
        __syncwarp();
      }
      // a scale's bits, so its exponent + 1 (fp16; subnormal ones are below 2^-14)
      const int high = (int)(__reduce_max_sync(0xffffffffu, big) >> 10) - 14;
      if (high > top) {
        const float f = pow2i(top - high);
        top = high;
#pragma unroll
        for (int r = 0; r < RT; ++r)
#pragma unroll
          for (int c = 0; c < 2 * NC; ++c)
#pragma unroll
            for (int e = 0; e < 4; ++e) o[r][c][e] *= f;
      }
      const float vscale = pow2i(-top);
      float f0[RT], f1[RT];  // what the rows 2 tq and 2 tq + 1 of the outputs are scaled by
#pragma unroll
      for (int r = 0; r < RT; ++r) {
        const float f = q[r].down * p.scale_log2;
        float mx = m[r];
#pragma unroll
        for (int n = 0; n < 4; ++n)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float x = s[r][n][e] * f;
            if (!all) {
              const int c = 8 * n + 2 * tq + e, j = k0 + c;
              const bool see = (okw >> c & 1u) && j <= pos[r] && (j >= lo[r] || j < p.sinks);
              x = see ? x : -INFINITY;
            }
            s[r][n][e] = x;
            mx = fmaxf(mx, x);
          }
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
        const float ref = mx == -INFINITY ? 0.f : mx - 14.f;
        const float down = mx == -INFINITY ? 0.f : fast_exp2(m[r] - mx);
        m[r] = mx;
        f0[r] = __shfl_sync(0xffffffffu, down, 8 * tq);
        f1[r] = __shfl_sync(0xffffffffu, down, 8 * tq + 4);
        l[r] *= down;
#pragma unroll
        for (int n = 0; n < 4; ++n)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            s[r][n][e] = fast_exp2(s[r][n][e] - ref);
            l[r] += s[r][n][e];
          }
      }
      const unsigned char *vrow = vt + lane * F::REC;
      uint32_t par[4];
      ldmatrix_x4_trans(par[0], par[1], par[2], par[3], vrow + F::CODES);
#pragma unroll
      for (int r = 0; r < RT; ++r) {
        float add[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int kb = 0; kb < 2; ++kb) {
          const uint32_t b0 = pack2<__half>(s[r][2 * kb][0], s[r][2 * kb][1]);
          const uint32_t b1 = pack2<__half>(s[r][2 * kb + 1][0], s[r][2 * kb + 1][1]);
          mma_16816<__half>(add, par[2 * kb], 0u, par[2 * kb + 1], 0u, b0, b1);
          if constexpr (SPLIT) {
            const float2 h0 = __half22float2(*reinterpret_cast<const __half2 *>(&b0));
            const float2 h1 = __half22float2(*reinterpret_cast<const __half2 *>(&b1));
            mma_16816<__half>(add, par[2 * kb], 0u, par[2 * kb + 1], 0u,
                              pack2<__half>(s[r][2 * kb][0] - h0.x, s[r][2 * kb][1] - h0.y),
                              pack2<__half>(s[r][2 * kb + 1][0] - h1.x, s[r][2 * kb + 1][1] - h1.y));
          }
        }
        if constexpr (MIDDLE) {  // (the lanes of the least values take those of the scales)
          const float x = __shfl_xor_sync(0xffffffffu, add[0], 16), y = __shfl_xor_sync(0xffffffffu, add[1], 16);
          add[0] = fmaf(8.f, x, add[0]);
          add[1] = fmaf(8.f, y, add[1]);
        }
        vmin[r][0] = fmaf(vmin[r][0], f0[r], add[0]);
        vmin[r][1] = fmaf(vmin[r][1], f1[r], add[1]);
      }
      float sc[4][2][4];  // scales of the lane's keys
#pragma unroll
      for (int n = 0; n < 4; ++n)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          q4_four(vt + (8 * n + 2 * tq + e) * F::REC + F::CODES, sc[n][e]);
#pragma unroll
          for (int g = 0; g < 4; ++g) sc[n][e][g] *= vscale;
        }
#pragma unroll
      for (int c = 0; c < NC; ++c) {
        uint32_t w[4], u[4][4];
        ldmatrix_x4_trans(w[0], w[1], w[2], w[3], vrow + c * 16);
#pragma unroll
        for (int i = 0; i < 4; ++i) q4_unpack(w[i], u[i]);
#pragma unroll
        for (int r = 0; r < RT; ++r) {
          uint32_t b[4], b2[4];  // p times scale, of the chunk's group (of each half's: D = 64)
          float from[4] = {0.f, 0.f, 0.f, 0.f};  // - 8 times their sums
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const int g = F::group_of(c, h);
            if (D == 64 || h == 0) {
#pragma unroll
              for (int n = 0; n < 4; ++n) {
                const float x = s[r][n][0] * sc[n][0][g], y = s[r][n][1] * sc[n][1][g];
                b[n] = pack2<__half>(x, y);
                if constexpr (SPLIT) {
                  const float2 hi = __half22float2(*reinterpret_cast<const __half2 *>(&b[n]));
                  b2[n] = pack2<__half>(x - hi.x, y - hi.y);
                }
              }
              if constexpr (MIDDLE) {
                constexpr uint32_t low = 0x80088008u, high = 0x80808080u;  // -8 2^-24, -8 2^-20
                from[0] = from[1] = from[2] = from[3] = 0.f;
#pragma unroll
                for (int kb = 0; kb < 2; ++kb) {
                  mma_16816<__half>(from, low, high, low, high, b[2 * kb], b[2 * kb + 1]);
                  if constexpr (SPLIT) mma_16816<__half>(from, low, high, low, high, b2[2 * kb], b2[2 * kb + 1]);
                }
              }
            }
            float add[4] = {from[0], from[1], from[2], from[3]};
#pragma unroll
            for (int kb = 0; kb < 2; ++kb) {
              mma_16816<__half>(add, u[2 * kb][2 * h], u[2 * kb][2 * h + 1], u[2 * kb + 1][2 * h],
                                u[2 * kb + 1][2 * h + 1], b[2 * kb], b[2 * kb + 1]);
              if constexpr (SPLIT)
                mma_16816<__half>(add, u[2 * kb][2 * h], u[2 * kb][2 * h + 1], u[2 * kb + 1][2 * h],
                                  u[2 * kb + 1][2 * h + 1], b2[2 * kb], b2[2 * kb + 1]);
            }
            o[r][2 * c + h][0] = fmaf(o[r][2 * c + h][0], f0[r], add[0]);
            o[r][2 * c + h][1] = fmaf(o[r][2 * c + h][1], f1[r], add[1]);
            o[r][2 * c + h][2] = fmaf(o[r][2 * c + h][2], f0[r], add[2]);
            o[r][2 * c + h][3] = fmaf(o[r][2 * c + h][3], f1[r], add[3]);
          }
        }
      }
      __syncwarp();  // the stage has been read
    }

    // ---- join the warps: each adds its part to the CTA's result in turn
    float f[RT];
#pragma unroll
    for (int r = 0; r < RT; ++r) {
      l[r] += __shfl_xor_sync(0xffffffffu, l[r], 1);
      l[r] += __shfl_xor_sync(0xffffffffu, l[r], 2);
      if (!ok) {
        m[r] = -INFINITY;
        l[r] = 0.f;
      }
      if (tq == 0) {
        sm.wm[warp][8 * r + gq] = m[r];
        sm.wl[warp][8 * r + gq] = l[r];
      }
    }
    __syncthreads();  // (and the result of an earlier piece has been read)
#pragma unroll
    for (int r = 0; r < RT; ++r) {
      float mr = -INFINITY, lr = 0.f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) mr = fmaxf(mr, sm.wm[w][8 * r + gq]);
#pragma unroll
      for (int w = 0; w < kWarps; ++w)
        if (sm.wm[w][8 * r + gq] != -INFINITY) lr = fmaf(sm.wl[w][8 * r + gq], fast_exp2(sm.wm[w][8 * r + gq] - mr), lr);
      f[r] = m[r] == -INFINITY ? 0.f : fast_exp2(m[r] - mr);
      if (warp == 0 && tq == 0) sm.ml[8 * r + gq] = make_float2(mr - 14.f, lr);  // (-inf: nothing seen)
    }
    for (int w = 0; w < kWarps; ++w) {
      if (warp == w && pc.t0 + w < pc.t1) {
#pragma unroll
        for (int r = 0; r < RT; ++r)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const float fr = __shfl_sync(0xffffffffu, f[r], 8 * tq + 4 * e);
            const float up = pow2i(24) * pow2i(top);
            float *res = sm.res + (8 * r + 2 * tq + e) * C::OP;
#pragma unroll
            for (int c = 0; c < NC; ++c)
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                const float low = __shfl_sync(0xffffffffu, vmin[r][e], 16 + 4 * F::group_of(c, h) + tq);
                const float x = fmaf(o[r][2 * c + h][e], up, low), y = fmaf(o[r][2 * c + h][2 + e], up * 0.0625f, low);
                float2 *at = reinterpret_cast<float2 *>(res + F::out_feature(c, h, gq));
                float2 v = w ? *at : make_float2(0.f, 0.f);
                v.x += fr == 0.f ? 0.f : x * fr;
                v.y += fr == 0.f ? 0.f : y * fr;
                *at = v;
              }
          }
      }
      __syncthreads();
    }
    if (!S) {
      for (int u = tid; u < po.rows * (D / 4); u += kThreads) {
        const int r = u / (D / 4), d = (u % (D / 4)) * 4;
        const float4 v = *reinterpret_cast<const float4 *>(sm.res + r * C::OP + d);
        const float x[4] = {v.x, v.y, v.z, v.w};
        const float2 ml = sm.ml[r];
        RowOut<T, D, ROWS>(p, po, r, ml.x, ml.y, d == 0).put(d, x);
      }
    }
  }
  // no copy may be in flight when the CTA exits, even if a wait gave up
  for (; used < put; ++used) mbar_wait(full + used % STAGES, (used / STAGES) & 1, p.err);
  if (S) join_cluster<T, D, ROWS, C::OP, kThreads>(p, pieces, sm.ml, sm.res);
}

template <typename T, int D, int RT>
mgqa_status launch_t(Q4Params qp, mgqa_dtype dt, const CacheAttnLaunch &how, cudaStream_t s) {
  using C = Cfg<D, RT>;
  auto kern = cache_q4_kernel<T, D, RT>;
  static std::atomic<uint64_t> attr{0};
  const mgqa_status st = ensure_cluster_attr(kern, C::smem, attr, "4-bit cache attention kernel");
  if (st != MGQA_OK) return st;
  CacheAttnParams &p = qp.t.a;
  p.block_rows = C::ROWS;
  p.RB = (p.R + C::ROWS - 1) / C::ROWS;
  p.tile_shift = kShift;
  const int64_t units = (int64_t)p.B * p.Hkv * p.RB;
  const int64_t tiles = most_tiles(p);
  qp.t.cluster = cluster_size(p, Q4<D>::REC, how.sms);
  if (qp.t.cluster) {
    const cudaError_t e = launch_pdl_cluster(kern, dim3((unsigned)(units * qp.t.cluster)), dim3(kThreads), C::smem, s,
                                             qp.t.cluster, qp);
    if (e != cudaSuccess) return fail(MGQA_ERR_CUDA, "4-bit cache attention launch: %s", cudaGetErrorString(e));
    return MGQA_OK;
  }
  p.lead = 8;
  p.min_run = 8;
  const int grid =
      (int)std::max<int64_t>(1, std::min<int64_t>(std::min(C::CTAS * how.sms, kMostCtas), units * (tiles + p.lead)));
  p.grid = grid;
  p.by_unit = units <= grid;
  p.cuts = static_cast<int4 *>(how.workspace);
  p.part_o = reinterpret_cast<float *>(p.cuts + kMostCtas);
  p.part_ml = reinterpret_cast<float2 *>(p.part_o + (size_t)2 * grid * C::ROWS * D);
  const cudaError_t e = launch_pdl(kern, dim3(grid), dim3(kThreads), C::smem, s, qp);
  if (e != cudaSuccess) return fail(MGQA_ERR_CUDA, "4-bit cache attention launch: %s", cudaGetErrorString(e));
  return launch_cache_merge(p, dt, D, C::ROWS, grid, s);
}

template <typename T, int D>
mgqa_status launch_d(const Q4Params &qp, mgqa_dtype dt, const CacheAttnLaunch &how, cudaStream_t s) {
  if (qp.t.a.R <= 8) return launch_t<T, D, 1>(qp, dt, how, s);
  return launch_t<T, D, 2>(qp, dt, how, s);
}

}  // namespace

// (of cache_attn_workspace_bytes)
static_assert(kMostCtas * 16 + (size_t)2 * kMostCtas * 32 * (128 + 2) * 4 <=
                  kCacheAttnMaxCtas * 16 + (size_t)kCacheAttnMaxCtas * 256 * (128 + 2) * 4,
              "the partial results fit in the workspace of the cache attention");

mgqa_status launch_attn_q4(const mgqa_args &a, const mgqa_pages *pages, int32_t window, int32_t sinks, void *ws,
                           cudaStream_t s) {
  Q4Params qp{};
  CacheAttnParams &p = qp.t.a;
  cache_attn_params(a, pages, nullptr, window, sinks, p);
  const CacheAttnLaunch how{ws, device_sm_count()};
  if (how.sms < 1) return fail(MGQA_ERR_CUDA, "cannot read the SM count of the current device");
  const int64_t rec = a.D / 2 + 16;
  qp.run_slots = p.ks[2] == rec && p.vs[2] == rec ? (p.table ? p.page_size : p.cap) : 1;
  if (a.dtype == MGQA_BF16)
    return a.D == 64 ? launch_d<__nv_bfloat16, 64>(qp, a.dtype, how, s) : launch_d<__nv_bfloat16, 128>(qp, a.dtype, how, s);
  if (a.dtype == MGQA_FP16)
    return a.D == 64 ? launch_d<__half, 64>(qp, a.dtype, how, s) : launch_d<__half, 128>(qp, a.dtype, how, s);
  return a.D == 64 ? launch_d<float, 64>(qp, a.dtype, how, s) : launch_d<float, 128>(qp, a.dtype, how, s);
}

}  // namespace mgqa
