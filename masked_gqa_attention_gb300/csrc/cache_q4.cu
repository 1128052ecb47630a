// Attention of the last T cached tokens of every request over a cache in 4 bits
// (cache_q4.cuh has the records and the products).
//
// Query t of request b, with n = kv_len[b], stands at position pos = n - T + t
// (below 0: it sees nothing) and sees slot j when
//   j <= pos and (no window, or pos - j < window, or j < sinks).
//
// Every visible record is read once per KV head and block of query rows, and takes a
// warp some 747 instructions per 32 keys of 128 features with 8 rows of queries, where
// the reads take 217 cycles of an SM. The latency of that work bounds it: three warps a
// scheduler issue 2.5 instructions a cycle of an SM's four, no pipe is half used, and a
// warp mostly waits for its own last instruction (32 requests of 16425 slots on average, 8
// KV heads of 4 query heads: 145 us, 0.68 of the copy rate; with 16 rows 216). Each warp
// streams tiles of 32 keys of its own through a ring in shared memory (cache_stream.cuh).
// The records are the first operand of both products (16 keys, or 16 features, by 8 rows
// of queries), so a code is unpacked once for all rows and no part of a product is empty
// with 8 rows (queries as the first operand took half as long again); the weights turn from
// one layout to the other by four transposes of 8 x 8 a tile. Long calls of more than 16
// rows take blocks of 32 (four heads by 8 tokens: 298 us, in blocks of 16 9 % more), which
// at D = 128 spill 304 bytes a thread to local memory, blocks of 16 72 (fp32 36), at two
// CTAs an SM; 8 rows spill none.
//
// Weights: p is 2^14 at most (the maximum is subtracted 14 short) and becomes fp16,
// 2^-11 of it down to 2^-28 of the largest; p times a scale is rounded once more.
// Scales of 2 and more are divided by a power of two first, which the outputs are in
// units of. fp32 calls hold both in two terms (2^-22). Sums of weights and outputs are
// fp32, a tile's from the tensor cores and those of the tiles in rounded additions:
// codes and least values are sums of one sign that nearly cancel, and the tensor
// cores' sums are truncated (with running accumulators 0.0066 of the outputs' size from
// 64 bits over 98000 keys). For the same reason the codes are taken from the middle c of
// the tile's group, where its values are about 0,
//   out_d = sum_j (p_j scale_jg) (u_jd - c) + sum_j p_j (least_jg + c scale_jg):
// the second rounding is one and the same for all keys of one weight and scale, does not
// average out, and would be multiplied by codes of one sign (100000 such keys: 0.05 of
// the outputs' size with codes from 0 and a mean code of 7.5, up to 0.11 with other means;
// from 8 instead of 7.5 still 0.004, and 0.07 where the mean is 2.5; so 0.0008). c is -sum least / sum scale
// of the tile's keys in steps of 1/64, so that u - c is exact and any c is right: 82 of
// the instructions (the batch above 138 us without; p times scale in two terms 153, the
// roundings summed and put right at the end 145, but with 32 rows 8 % more than this).
//
// The work is cut as for the other cache attention (cache_sched.cuh): equal runs of
// tiles and the merge kernel for long calls, a cluster per unit for short ones.
#include <algorithm>
#include <cmath>

#include "cache_q4.cuh"
#include "cache_stream.cuh"

namespace mgqa {
namespace {

constexpr int kWarps = 4;
constexpr int kThreads = 32 * kWarps;
constexpr int kShift = 5, kKeys = 32;  // keys of a tile
constexpr float kNothing = -3.4028235e38f;  // the maximum of a row that has seen nothing (no score is below it)
constexpr int kMostCtas = 512;  // partial results: two per CTA

template <int D, int RT>
struct Cfg {
  static constexpr int ROWS = 8 * RT;
  static constexpr int STAGES = 2;
  static constexpr int CTAS = RT == 1 ? 3 : 2;  // of an SM
  static constexpr int TILEB = kKeys * Q4<D>::REC;
  static constexpr int ring = kWarps * STAGES * 2 * TILEB;
  static constexpr int OP = D + 4;  // row pitch of a CTA's result (floats)
  struct Misc {
    float res[ROWS * OP];             // the CTA's result, 16-byte aligned
    float wm[kWarps][ROWS], wl[kWarps][ROWS];
    float2 ml[ROWS];
    LocateScratch<kThreads> scratch;
    int2 what[kWarps][STAGES];        // a stage's first slot, and which keys count
    Feed feed[kWarps];
    // with four groups of rows: their operands (the products', then the sums), and of
    // each row the scores' factor and the position
    uint2 q[RT == kWarps ? RT : 1][RT == kWarps ? 4 * Q4<D>::KS + 1 : 1][32];
    float2 rule[ROWS];
  };
  static constexpr int smem = ring + (int)sizeof(Misc);
};

template <typename T, int D, int RT>
__global__ void __launch_bounds__(kThreads, (Cfg<D, RT>::CTAS))
cache_q4_kernel(const __grid_constant__ StreamParams qp) {
  using C = Cfg<D, RT>;
  using F = Q4<D>;
  constexpr bool SPLIT = sizeof(T) == 4;
  constexpr int ROWS = C::ROWS, STAGES = C::STAGES, NC = F::CHUNKS;
  constexpr bool SHARE = RT == kWarps;
  static_assert(!SHARE || !SPLIT, "one term of the queries is staged");
  const CacheAttnParams &p = qp.t.a;
  extern __shared__ __align__(1024) unsigned char smem[];
  auto &sm = *reinterpret_cast<typename C::Misc *>(smem + C::ring);
  const int tid = threadIdx.x, lane = lane_id(), warp = tid >> 5, gq = lane >> 2, tq = lane & 3;
  unsigned char *ring = smem + warp * (STAGES * 2 * C::TILEB);
  if (warp == 1) touch_params(qp, lane);
  grid_dependency_wait();
  allow_dependents();
  Pieces pieces{};
  pieces.start<kThreads>(qp.t, sm.scratch);
  const int S = pieces.S;
  const bool teller = tid == 0 && !S;
  if (teller) tell_cut(p, blockIdx.x, nullptr);

  Stream<kKeys, F::REC / 16, kAsIs, true, kWarps> ahead(sm.feed[warp], 1);
  ahead.start(qp, pieces, warp, lane);
  int put = 0, st = 0;  // stages: filled next, used next
  const auto start_one = [&] {
    if (ahead.live) {
      ahead.issue(qp, warp, lane, ring + put * 2 * C::TILEB, sm.what[warp] + put);
      put = put + 1 == STAGES ? 0 : put + 1;
    }
    cp_async_commit();
  };
  for (int s = 0; s < STAGES - 1; ++s) start_one();

  if (pieces.idle())
    for (int r = tid; r < ROWS; r += kThreads) sm.ml[r] = make_float2(-INFINITY, 0.f);  // no share of the unit
  Piece pc;
  while (pieces.next(p, pc)) {
    if (teller) tell_cut(p, blockIdx.x, &pc);
    const RowPlan &rp = pc.rp;
    const PieceOut po = out_of(p, pc, blockIdx.x);
    // of the rows 2 tq and 2 tq + 1 of each group, whose scores and outputs the lane has
    float scale[RT][2];
    int pos[RT][2];
    Q4Row<D, SPLIT> q[SHARE ? 1 : RT];  // (four groups: staged in shared memory, one by each warp)
    const auto load_row = [&](int r, Q4Row<D, SPLIT> &to) {  // its position
      const int row = po.row0 + 8 * r + gq;
      const bool in = row < p.R;
      const int t = in ? row / p.n_rep : 0, h = pc.g * p.n_rep + (in ? row - t * p.n_rep : 0);
      to.load(in ? static_cast<const T *>(p.q) + (int64_t)pc.b * p.qs[0] + (int64_t)h * p.qs[1] + (int64_t)t * p.qs[2]
                 : static_cast<const T *>(nullptr), tq, p.scale_log2 < 0.f);
      return in ? rp.n - p.T + t : -1;
    };
    // (above 0, so that a hidden key's -inf stays one)
    const auto factor = [&](float down) { return fmaxf(down * fabsf(p.scale_log2), 1.2e-38f); };
    if constexpr (SHARE) {
      const int at = load_row(warp, q[0]);
      if (tq == 0) sm.rule[8 * warp + gq] = make_float2(factor(q[0].down), __int_as_float(at));
#pragma unroll
      for (int g = 0; g < 4; ++g)
#pragma unroll
        for (int i = 0; i < F::KS; ++i) sm.q[warp][g * F::KS + i][lane] = make_uint2(q[0].a[g][i][0], q[0].a[g][i][1]);
      sm.q[warp][4 * F::KS][lane] = make_uint2(q[0].sums[0], q[0].sums[1]);
      __syncthreads();
#pragma unroll
      for (int r = 0; r < RT; ++r)
#pragma unroll
        for (int e = 0; e < 2; ++e) scale[r][e] = sm.rule[8 * r + 2 * tq + e].x;
    } else {
#pragma unroll
      for (int r = 0; r < RT; ++r) {
        const int at = load_row(r, q[r]);
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          scale[r][e] = factor(__shfl_sync(0xffffffffu, q[r].down, 8 * tq + 4 * e));
          pos[r][e] = __shfl_sync(0xffffffffu, at, 8 * tq + 4 * e);
        }
      }
    }
    // every row of the block sees the keys from `far` (and the sinks) to `near`
    const int near = rp.n - p.T + po.row0 / p.n_rep;
    const int far = rp.n - p.T + (po.row0 + po.rows - 1) / p.n_rep - p.window + 1;

    float o[RT][2 * NC][4], vmin[RT][2], m[RT][2], l[RT][2];
    int top = SPLIT ? -30 : 0;  // outputs are in units of 2^top (see below)
#pragma unroll
    for (int r = 0; r < RT; ++r) {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        m[r][e] = kNothing;
        l[r][e] = vmin[r][e] = 0.f;
      }
#pragma unroll
      for (int c = 0; c < 2 * NC; ++c) o[r][c][0] = o[r][c][1] = o[r][c][2] = o[r][c][3] = 0.f;
    }
    for (int t = pc.t0 + warp; t < pc.t1; t += kWarps) {
      start_one();
      cp_async_wait<STAGES - 1>();
      __syncwarp();
      const unsigned char *kt = ring + st * 2 * C::TILEB;
      unsigned char *vt = ring + (st * 2 + 1) * C::TILEB;
      const int k0 = sm.what[warp][st].x;
      const uint32_t okw = (uint32_t)sm.what[warp][st].y;
      const unsigned char *krow = kt + lane * F::REC;
      unsigned char *vrow = vt + lane * F::REC;

      // ---- scores: keys 16 i + gq and 16 i + 8 + gq
      Q4Scores<D, SPLIT> x[RT][2];
      {
#pragma unroll
        for (int i = 0; i < 2; ++i) {  // (the two halves of the first operand's columns are the same parameters)
          uint32_t par[4];
          ldmatrix_x4(par[0], par[1], par[2], par[3], kt + (16 * i + (lane & 15)) * F::REC + F::CODES);
#pragma unroll
          for (int r = 0; r < RT; ++r) {
            if constexpr (SHARE) {
              const uint2 both = sm.q[r][4 * F::KS][lane];
              const uint32_t sums[2] = {both.x, both.y};
              x[r][i].least(par, sums);
            } else {
              x[r][i].least(par, q[r].sums);
            }
          }
        }
        float sc[4][4];
#pragma unroll
        for (int i = 0; i < 4; ++i) q4_four(kt + (8 * i + gq) * F::REC + F::CODES, sc[i]);
#pragma unroll
        for (int c = 0; c < NC; ++c) {
          uint32_t w[4];
          ldmatrix_x4(w[0], w[1], w[2], w[3], krow + c * 16);
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            uint32_t u[2][4];
            q4_codes<SPLIT>(w[2 * i], u[0]);
            q4_codes<SPLIT>(w[2 * i + 1], u[1]);
            const float(&two)[2][4] = reinterpret_cast<const float(&)[2][4]>(sc[2 * i]);
#pragma unroll
            for (int r = 0; r < RT; ++r)
              x[r][i].chunk(c, u, two,
                            [&](int g, int s) {
                              if constexpr (SHARE) return sm.q[r][g * F::KS + s][lane];
                              else return make_uint2(q[r].a[g][s][0], q[r].a[g][s][1]);
                            },
                            [&](int g, int s) {
                              const auto &row = q[SHARE ? 0 : r];
                              return make_uint2(row.b[SPLIT ? g : 0][s][0], row.b[SPLIT ? g : 0][s][1]);
                            });
          }
        }
#pragma unroll
        for (int r = 0; r < RT; ++r)
#pragma unroll
          for (int i = 0; i < 2; ++i) x[r][i].finish();
      }

      // ---- the largest scale of V: its bits give an exponent, every scale is below 2^high
      const uint2 vsc = *reinterpret_cast<const uint2 *>(vrow + F::CODES);
      uint32_t big = __vmaxu2(vsc.x, vsc.y);
      big = max(big & 0xffffu, big >> 16);
      const int high = (int)(__reduce_max_sync(0xffffffffu, big) >> 10) - 14;
      if (high > (SPLIT ? top : max(top, 1))) {
        const float f = pow2i(top - high);
        top = high;
#pragma unroll
        for (int r = 0; r < RT; ++r)
#pragma unroll
          for (int c = 0; c < 2 * NC; ++c)
#pragma unroll
            for (int e = 0; e < 4; ++e) o[r][c][e] *= f;
      }

      // ---- the parameters of V: lane (g, tq) has the scales of group g of two keys, lane
      // (4 + g, tq) their least values: keys 2 tq and + 1 behind 0, 16, 8 and 24. So both
      // halves of the keys are in one operand, above and below (of each product one half
      // of the rows is of no use). And in the lanes of the least values the middle of the
      // group's codes, as a number and as the pair -middle 2^-9.
      uint32_t vpar[4], minus;
      float middle;
      const auto look = [&] {
        ldmatrix_x4_trans(vpar[0], vpar[1], vpar[2], vpar[3],
                          vt + ((lane & 7) | (lane & 8) << 1 | (lane & 16) >> 1) * F::REC + F::CODES);
        constexpr uint32_t one = 0x3c003c00u;
        float sums[4];
        mma_16816_first<__half>(sums, vpar[0], vpar[1], vpar[2], vpar[3], one, one);
        const float mine = sums[0] + sums[2], across = __shfl_xor_sync(0xffffffffu, mine, 16);
        const float c = fminf(fmaxf(__fdividef(-mine, across), 0.f), 15.f);  // (0 / 0: 0)
        middle = __fsub_rn(__fadd_rn(c, 196608.f), 196608.f);                 // 1.5 2^17: steps of 1/64
        minus = pack2<__half>(middle * -0x1p-9f, middle * -0x1p-9f);
      };
      // (four groups of rows: ahead of the weights, which hide its latency: 64 tokens a
      // request 5 % faster; with one group the registers are worth more, 1 %)
      if constexpr (SHARE) look();

      // ---- weights, and their transpose: pw[r][n] has row gq, keys 8 n + 2 tq and + 1
      const bool all = okw == 0xffffffffu && k0 + kKeys - 1 <= near && (k0 >= far || k0 + kKeys <= p.sinks);
      if (!all) {
#pragma unroll
        for (int r = 0; r < RT; ++r)
#pragma unroll
          for (int n = 0; n < 4; ++n)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const int c = 8 * n + gq, j = k0 + c;
              const int at = SHARE ? __float_as_int(sm.rule[8 * r + 2 * tq + e].y) : pos[r][e];
              const bool see = (okw >> c & 1u) && j <= at && (j > at - p.window || j < p.sinks);
              float &s = x[r][n / 2].s[n % 2 * 2 + e];
              s = see ? s : -INFINITY;
            }
      }
      uint32_t pw[RT][4], pw2[SPLIT ? RT : 1][4];
      float down[RT][2];
#pragma unroll
      for (int r = 0; r < RT; ++r) {
        float ref[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float mx = fmaxf(fmaxf(x[r][0].s[e], x[r][0].s[2 + e]), fmaxf(x[r][1].s[e], x[r][1].s[2 + e]));
          mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 4));
          mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 8));
          mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 16));
          mx = fmaxf(m[r][e], __fmul_rn(mx, scale[r][e]));
          ref[e] = mx - 14.f;
          down[r][e] = fast_exp2(m[r][e] - mx);
          m[r][e] = mx;
          l[r][e] *= down[r][e];
        }
#pragma unroll
        for (int n = 0; n < 4; ++n) {
          float *s = x[r][n / 2].s + n % 2 * 2;
          // (rounded as the maximum was: of huge scores only equal ones cancel)
          s[0] = fast_exp2(__fsub_rn(__fmul_rn(s[0], scale[r][0]), ref[0]));
          s[1] = fast_exp2(__fsub_rn(__fmul_rn(s[1], scale[r][1]), ref[1]));
          l[r][0] += s[0];
          l[r][1] += s[1];
          const uint32_t w = pack2<__half>(s[0], s[1]);
          pw[r][n] = movmatrix_trans(w);
          if constexpr (SPLIT) {
            const float2 hi = __half22float2(*reinterpret_cast<const __half2 *>(&w));
            pw2[r][n] = movmatrix_trans(pack2<__half>(s[0] - hi.x, s[1] - hi.y));
          }
        }
      }

      // ---- outputs
      if constexpr (!SHARE) look();
      {
        uint32_t vmin1[4], vmin2[4];  // (fp32: least + middle scale, in two terms, in the lanes of the least values)
#pragma unroll
        for (int n = 0; n < 4; ++n) {
          vmin1[n] = vpar[n];
          if constexpr (SPLIT) {
            const uint32_t across = __shfl_xor_sync(0xffffffffu, vpar[n], 16);
            const float2 least = __half22float2(*reinterpret_cast<const __half2 *>(&vpar[n]));
            const float2 scale2 = __half22float2(*reinterpret_cast<const __half2 *>(&across));
            const float y = fmaf(middle, scale2.x, least.x), z = fmaf(middle, scale2.y, least.y);
            vmin1[n] = pack2<__half>(y, z);
            const float2 got = __half22float2(*reinterpret_cast<const __half2 *>(&vmin1[n]));
            vmin2[n] = pack2<__half>(y - got.x, z - got.y);
          }
        }
#pragma unroll
        for (int r = 0; r < RT; ++r) {
          float add[4], behind[4];
          mma_16816_first<__half>(add, vmin1[0], vmin1[1], vmin1[2], vmin1[3], pw[r][0], pw[r][1]);
          mma_16816_first<__half>(behind, vmin1[0], vmin1[1], vmin1[2], vmin1[3], pw[r][2], pw[r][3]);
          if constexpr (SPLIT) {
            mma_16816<__half>(add, vmin1[0], vmin1[1], vmin1[2], vmin1[3], pw2[r][0], pw2[r][1]);
            mma_16816<__half>(behind, vmin1[0], vmin1[1], vmin1[2], vmin1[3], pw2[r][2], pw2[r][3]);
            mma_16816<__half>(add, vmin2[0], vmin2[1], vmin2[2], vmin2[3], pw[r][0], pw[r][1]);
            mma_16816<__half>(behind, vmin2[0], vmin2[1], vmin2[2], vmin2[3], pw[r][2], pw[r][3]);
          }
          add[0] += behind[2];
          add[1] += behind[3];
          if constexpr (!SPLIT) {  // (the lanes of the least values take those of the scales)
            const float a = __shfl_xor_sync(0xffffffffu, add[0], 16), b = __shfl_xor_sync(0xffffffffu, add[1], 16);
            add[0] = fmaf(middle, a, add[0]);
            add[1] = fmaf(middle, b, add[1]);
          }
          vmin[r][0] = fmaf(vmin[r][0], down[r][0], add[0]);
          vmin[r][1] = fmaf(vmin[r][1], down[r][1], add[1]);
        }
      }
      uint32_t sc[4][4];  // scales of keys 8 n + 2 tq and + 1, by groups
#pragma unroll
      for (int g = 0; g < 4; ++g)
#pragma unroll
        for (int n = 0; n < 4; ++n) sc[g][n] = __shfl_sync(0xffffffffu, vpar[(n & 1) << 1 | n >> 1], 4 * g + tq);
      if (!SPLIT && top != 0) {
        const __half2 f = __float2half2_rn(pow2i(-top));
#pragma unroll
        for (int g = 0; g < 4; ++g)
#pragma unroll
          for (int n = 0; n < 4; ++n) {
            const __half2 y = __hmul2(*reinterpret_cast<const __half2 *>(&sc[g][n]), f);
            sc[g][n] = *reinterpret_cast<const uint32_t *>(&y);
          }
      }
      const float unit = pow2i(-top);
#pragma unroll
      for (int c = 0; c < NC; ++c) {
        uint32_t w[4], u[4][4], from[2];  // from: minus the middle of each half's group
#pragma unroll
        for (int h = 0; h < 2; ++h)
          from[h] = D == 128 && h ? from[0] : __shfl_sync(0xffffffffu, minus, 16 + 4 * F::group_of(c, h));
        ldmatrix_x4_trans(w[0], w[1], w[2], w[3], vrow + c * 16);
#pragma unroll
        for (int n = 0; n < 4; ++n) q4_unpack_from(w[n], from, u[n]);
#pragma unroll
        for (int r = 0; r < RT; ++r) {
          uint32_t b[4], b2[4];  // weight times scale, of the chunk's group (of each half's: D = 64)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const int g = F::group_of(c, h);
            if (D == 64 || h == 0) {
#pragma unroll
              for (int n = 0; n < 4; ++n) {
                const __half2 s2 = *reinterpret_cast<const __half2 *>(&sc[g][n]), p2 = *reinterpret_cast<const __half2 *>(&pw[r][n]);
                if constexpr (SPLIT) {
                  const float2 hi = __half22float2(p2), lo = __half22float2(*reinterpret_cast<const __half2 *>(&pw2[r][n]));
                  const float2 sf = __half22float2(s2);
                  const float y = (hi.x + lo.x) * (sf.x * unit), z = (hi.y + lo.y) * (sf.y * unit);
                  b[n] = pack2<__half>(y, z);
                  const float2 got = __half22float2(*reinterpret_cast<const __half2 *>(&b[n]));
                  b2[n] = pack2<__half>(y - got.x, z - got.y);
                } else {
                  const __half2 y = __hmul2(p2, s2);
                  b[n] = *reinterpret_cast<const uint32_t *>(&y);
                }
              }
            }
            float add[4];
            mma_16816_first<__half>(add, u[0][2 * h], u[0][2 * h + 1], u[1][2 * h], u[1][2 * h + 1], b[0], b[1]);
            mma_16816<__half>(add, u[2][2 * h], u[2][2 * h + 1], u[3][2 * h], u[3][2 * h + 1], b[2], b[3]);
            if constexpr (SPLIT) {
              mma_16816<__half>(add, u[0][2 * h], u[0][2 * h + 1], u[1][2 * h], u[1][2 * h + 1], b2[0], b2[1]);
              mma_16816<__half>(add, u[2][2 * h], u[2][2 * h + 1], u[3][2 * h], u[3][2 * h + 1], b2[2], b2[3]);
            }
            float(&to)[4] = o[r][2 * c + h];
            to[0] = fmaf(to[0], down[r][0], add[0]);
            to[1] = fmaf(to[1], down[r][1], add[1]);
            to[2] = fmaf(to[2], down[r][0], add[2]);
            to[3] = fmaf(to[3], down[r][1], add[3]);
          }
        }
      }
      __syncwarp();  // the stage has been read
      st = st + 1 == STAGES ? 0 : st + 1;
    }

    // ---- join the warps: each adds its part to the CTA's result in turn
    float f[RT][2];
#pragma unroll
    for (int r = 0; r < RT; ++r)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        l[r][e] += __shfl_xor_sync(0xffffffffu, l[r][e], 4);
        l[r][e] += __shfl_xor_sync(0xffffffffu, l[r][e], 8);
        l[r][e] += __shfl_xor_sync(0xffffffffu, l[r][e], 16);
        if (m[r][e] == kNothing) m[r][e] = -INFINITY;
        if (gq == 0) {
          sm.wm[warp][8 * r + 2 * tq + e] = m[r][e];
          sm.wl[warp][8 * r + 2 * tq + e] = l[r][e];
        }
      }
    __syncthreads();  // (and the result of an earlier piece has been read)
#pragma unroll
    for (int r = 0; r < RT; ++r)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int row = 8 * r + 2 * tq + e;
        float mr = -INFINITY, lr = 0.f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) mr = fmaxf(mr, sm.wm[w][row]);
#pragma unroll
        for (int w = 0; w < kWarps; ++w)
          if (sm.wm[w][row] != -INFINITY) lr = fmaf(sm.wl[w][row], fast_exp2(sm.wm[w][row] - mr), lr);
        f[r][e] = m[r][e] == -INFINITY ? 0.f : fast_exp2(m[r][e] - mr);
        if (warp == 0 && gq == 0) sm.ml[row] = make_float2(mr - 14.f, lr);  // (-inf: nothing seen)
      }
    for (int w = 0; w < kWarps; ++w) {
      if (warp == w && pc.t0 + w < pc.t1) {
        const float up = pow2i(9) * pow2i(top);
#pragma unroll
        for (int r = 0; r < RT; ++r)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float *res = sm.res + (8 * r + 2 * tq + e) * C::OP;
#pragma unroll
            for (int c = 0; c < NC; ++c)
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                const float low = __shfl_sync(0xffffffffu, vmin[r][e], 16 + 4 * F::group_of(c, h) + tq);
                const float y = fmaf(o[r][2 * c + h][e], up, low), z = fmaf(o[r][2 * c + h][2 + e], up, low);
                float2 *at = reinterpret_cast<float2 *>(res + F::out_feature(c, h, gq));
                float2 v = w ? *at : make_float2(0.f, 0.f);
                v.x += f[r][e] == 0.f ? 0.f : y * f[r][e];
                v.y += f[r][e] == 0.f ? 0.f : z * f[r][e];
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
  if (S) join_cluster<T, D, ROWS, C::OP, kThreads>(p, pieces, sm.ml, sm.res);
}

template <typename T, int D, int RT>
mgqa_status launch_t(StreamParams qp, mgqa_dtype dt, const CacheAttnLaunch &how, cudaStream_t s) {
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
mgqa_status launch_d(const StreamParams &qp, mgqa_dtype dt, const CacheAttnLaunch &how, cudaStream_t s) {
  if (qp.t.a.R <= 8) return launch_t<T, D, 1>(qp, dt, how, s);
  // (blocks of 32 rows cost less to unpack for, but a short call leaves SMs without one)
  if constexpr (sizeof(T) == 2)
    if (qp.t.a.R > 16 && !short_call(qp.t.a, Q4<D>::REC)) return launch_t<T, D, 4>(qp, dt, how, s);
  return launch_t<T, D, 2>(qp, dt, how, s);
}

}  // namespace

// (of cache_attn_workspace_bytes)
static_assert(kMostCtas * 16 + (size_t)2 * kMostCtas * 32 * (128 + 2) * 4 <=
                  kCacheAttnMaxCtas * 16 + (size_t)kCacheAttnMaxCtas * 256 * (128 + 2) * 4,
              "the partial results fit in the workspace of the cache attention");

mgqa_status launch_attn_q4(const mgqa_args &a, const mgqa_pages *pages, int32_t window, int32_t sinks, void *ws,
                           cudaStream_t s) {
  StreamParams qp{};
  CacheAttnParams &p = qp.t.a;
  cache_attn_params(a, pages, nullptr, window, sinks, p);
  const CacheAttnLaunch how{ws, device_sm_count()};
  if (how.sms < 1) return fail(MGQA_ERR_CUDA, "cannot read the SM count of the current device");
  if (!set_steps(qp, p.ks, p.vs, a.D / 2 + 16, pages ? pages->page_size : 0))
    return fail(MGQA_ERR_UNSUPPORTED, "strides of records past 2^36 bytes");
  if (a.dtype == MGQA_BF16)
    return a.D == 64 ? launch_d<__nv_bfloat16, 64>(qp, a.dtype, how, s) : launch_d<__nv_bfloat16, 128>(qp, a.dtype, how, s);
  if (a.dtype == MGQA_FP16)
    return a.D == 64 ? launch_d<__half, 64>(qp, a.dtype, how, s) : launch_d<__half, 128>(qp, a.dtype, how, s);
  return a.D == 64 ? launch_d<float, 64>(qp, a.dtype, how, s) : launch_d<float, 128>(qp, a.dtype, how, s);
}

}  // namespace mgqa
