// What the last T cached tokens look at: the attention weights that they give to
// every slot of the cache, summed over the tokens and over the query heads of a KV
// head, and added to what earlier calls have found:
//   weight[b,g,j] += sum_{t, h in g} exp(scale <q[b,h,t], k[b,g,j]> - lse[b,h,t])
// over the slots j that token t sees (the rule of cache_q4.cu); lse comes from the
// attention call.
//
// Every visible key is read once, 2 D operations for each of R = T Hq / Hkv rows:
// up to some 64 rows the reads bound it. Keys are independent of one another, so a
// warp takes 16 of them at a time straight into registers, as the first operand of
// m16n8k16 products with 8 rows of queries each from shared memory: a quad of lanes
// has a key, and each of its lanes the 16-byte pieces 4 i + its place, which is an
// order of the features that the queries are staged in too, so nothing is shuffled.
// The next 16 keys are on their way meanwhile. fp32 keys take the same places and
// the CUDA cores; keys in 4 bits the products of cache_q4.cuh.
//
// The tiles of all requests and KV heads are cut into equal runs (cache_sched.cuh);
// no sum crosses a warp but a quad's, so results repeat bit for bit.
#include <algorithm>

#include "cache_producer.cuh"
#include "cache_q4.cuh"

namespace mgqa {
namespace {

constexpr int kWarps = 4;
constexpr int kThreads = 32 * kWarps;
constexpr int kShift = 4, kKeys = 16;  // keys of a tile
constexpr int kChunkRows = 128;        // query rows that are staged at a time

struct WeightParams {
  TmaParams t;
  float *weight;
  int64_t ws[2];  // request, KV head
  int32_t chunk;  // rows staged at a time: a multiple of 8
};

// The keys gq and gq + 8 of a tile, as a lane holds them: 16-bit ...
template <typename T, int D>
struct Keys {
  using Query = T;
  static constexpr int N = D / 32;
  static constexpr int ROWB = D * (int)sizeof(T);
  static constexpr int STAGED = N * 512;  // bytes of 8 staged rows
  uint4 k[2][N];

  MGQA_DEV void load(int i, const char *row, int tq) {
#pragma unroll
    for (int c = 0; c < N; ++c) k[i][c] = __ldcs(reinterpret_cast<const uint4 *>(row) + 4 * c + tq);
  }
  MGQA_DEV void clear(int i) {
#pragma unroll
    for (int c = 0; c < N; ++c) k[i][c] = make_uint4(0u, 0u, 0u, 0u);
  }
  // Query row (null: zeros) of this lane's quad to its place of 8 staged rows; the
  // factor that its scores still need.
  static MGQA_DEV float stage(const T *row, unsigned char *to, int lane) {
#pragma unroll
    for (int c = 0; c < N; ++c)
      reinterpret_cast<uint4 *>(to)[c * 32 + lane] =
          row ? *(reinterpret_cast<const uint4 *>(row) + 4 * c + (lane & 3)) : make_uint4(0u, 0u, 0u, 0u);
    return 1.f;
  }
  // s: key gq, rows 2 tq and 2 tq + 1; key gq + 8
  MGQA_DEV void scores(const unsigned char *staged, int lane, float (&s)[4]) const {
#pragma unroll
    for (int c = 0; c < N; ++c) {
      const uint4 q = reinterpret_cast<const uint4 *>(staged)[c * 32 + lane];
      if (c == 0) mma_16816_first<T>(s, k[0][c].x, k[1][c].x, k[0][c].y, k[1][c].y, q.x, q.y);
      else mma_16816<T>(s, k[0][c].x, k[1][c].x, k[0][c].y, k[1][c].y, q.x, q.y);
      mma_16816<T>(s, k[0][c].z, k[1][c].z, k[0][c].w, k[1][c].w, q.z, q.w);
    }
  }
};

// ... 32-bit, on the CUDA cores ...
template <int D>
struct Keys<float, D> {
  using Query = float;
  static constexpr int N = D / 16;
  static constexpr int ROWB = D * 4;
  static constexpr int STAGED = 8 * D * 4;
  float4 k[2][N];

  MGQA_DEV void load(int i, const char *row, int tq) {
#pragma unroll
    for (int c = 0; c < N; ++c) k[i][c] = __ldcs(reinterpret_cast<const float4 *>(row) + 4 * c + tq);
  }
  MGQA_DEV void clear(int i) {
#pragma unroll
    for (int c = 0; c < N; ++c) k[i][c] = make_float4(0.f, 0.f, 0.f, 0.f);
  }
  static MGQA_DEV float stage(const float *row, unsigned char *to, int lane) {
#pragma unroll
    for (int c = 0; c < N; ++c)
      reinterpret_cast<float4 *>(to)[(lane >> 2) * (D / 4) + 4 * c + (lane & 3)] =
          row ? *(reinterpret_cast<const float4 *>(row) + 4 * c + (lane & 3)) : make_float4(0.f, 0.f, 0.f, 0.f);
    return 1.f;
  }
  MGQA_DEV void scores(const unsigned char *staged, int lane, float (&s)[4]) const {
    const int tq = lane & 3;
    s[0] = s[1] = s[2] = s[3] = 0.f;
#pragma unroll
    for (int r = 0; r < 8; ++r) {
      const float4 *q = reinterpret_cast<const float4 *>(staged) + r * (D / 4) + tq;
      float x = 0.f, y = 0.f;
#pragma unroll
      for (int c = 0; c < N; ++c) {
        const float4 f = q[4 * c];
        x = fmaf(k[0][c].x, f.x, x); x = fmaf(k[0][c].y, f.y, x);
        x = fmaf(k[0][c].z, f.z, x); x = fmaf(k[0][c].w, f.w, x);
        y = fmaf(k[1][c].x, f.x, y); y = fmaf(k[1][c].y, f.y, y);
        y = fmaf(k[1][c].z, f.z, y); y = fmaf(k[1][c].w, f.w, y);
      }
      x += __shfl_xor_sync(0xffffffffu, x, 1);
      y += __shfl_xor_sync(0xffffffffu, y, 1);
      x += __shfl_xor_sync(0xffffffffu, x, 2);
      y += __shfl_xor_sync(0xffffffffu, y, 2);
      if (tq == r / 2) {
        s[r % 2] = x;
        s[2 + r % 2] = y;
      }
    }
  }
};

// ... or in 4 bits, for queries of type T.
template <typename T, int D>
struct Q4Keys {
  using Query = T;
  using F = Q4<D>;
  static constexpr bool SPLIT = sizeof(T) == 4;
  static constexpr int N = F::CHUNKS;
  static constexpr int ROWB = F::REC;
  static constexpr int WORDS = 8 * F::KS;  // operand registers of a row, one term
  static constexpr int STAGED = (WORDS * (SPLIT ? 2 : 1) + 2) * 128;
  uint32_t k[2][N];
  uint4 par[2];

  MGQA_DEV void load(int i, const char *row, int tq) {
#pragma unroll
    for (int c = 0; c < N; ++c) k[i][c] = __ldg(reinterpret_cast<const uint32_t *>(row) + 4 * c + tq);
    par[i] = __ldg(reinterpret_cast<const uint4 *>(row + F::CODES));
  }
  MGQA_DEV void clear(int i) {
#pragma unroll
    for (int c = 0; c < N; ++c) k[i][c] = 0u;
    par[i] = make_uint4(0u, 0u, 0u, 0u);
  }
  static MGQA_DEV float stage(const T *row, unsigned char *to, int lane) {
    Q4Row<D, SPLIT> q;
    q.load(row, lane & 3);
    uint32_t *w = reinterpret_cast<uint32_t *>(to);
#pragma unroll
    for (int g = 0; g < 4; ++g)
#pragma unroll
      for (int i = 0; i < F::KS; ++i) {
        const int at = (g * F::KS + i) * 64 + 2 * lane;
        *reinterpret_cast<uint2 *>(w + at) = make_uint2(q.a[g][i][0], q.a[g][i][1]);
        if constexpr (SPLIT) *reinterpret_cast<uint2 *>(w + WORDS * 32 + at) = make_uint2(q.b[g][i][0], q.b[g][i][1]);
      }
    *reinterpret_cast<uint2 *>(w + (STAGED / 4 - 64) + 2 * lane) = make_uint2(q.sums[0], q.sums[1]);
    return q.down;
  }
  static MGQA_DEV void scales(const uint4 &p, float (&f)[4]) {
    const float2 a = __half22float2(*reinterpret_cast<const __half2 *>(&p.x));
    const float2 b = __half22float2(*reinterpret_cast<const __half2 *>(&p.y));
    f[0] = a.x; f[1] = a.y; f[2] = b.x; f[3] = b.y;
  }
  static MGQA_DEV uint32_t word(const uint4 &p, int tq) { return tq < 2 ? (tq ? p.y : p.x) : (tq == 2 ? p.z : p.w); }
  MGQA_DEV void scores(const unsigned char *staged, int lane, float (&s)[4]) const {
    const uint32_t *w = reinterpret_cast<const uint32_t *>(staged);
    const uint2 q = *reinterpret_cast<const uint2 *>(w + (STAGED / 4 - 64) + 2 * lane);
    const uint32_t sums[2] = {q.x, q.y};
    float sc[2][4];
    scales(par[0], sc[0]);
    scales(par[1], sc[1]);
    Q4Scores<D, SPLIT> x;
    const uint32_t p0 = word(par[0], lane & 3), p1 = word(par[1], lane & 3), both[4] = {p0, p1, p0, p1};
    x.least(both, sums);
    const auto term = [&](int t) {
      return [=](int g, int i) {
        return *reinterpret_cast<const uint2 *>(w + t * WORDS * 32 + (g * F::KS + i) * 64 + 2 * lane);
      };
    };
#pragma unroll
    for (int c = 0; c < N; ++c) {
      uint32_t u[2][4];
      q4_unpack(k[0][c], u[0]);
      q4_unpack(k[1][c], u[1]);
      x.chunk(c, u, sc, term(0), term(1));
    }
    x.finish();
#pragma unroll
    for (int e = 0; e < 4; ++e) s[e] = x.s[e];
  }
};

// Positions of the lane's two keys of a tile and their pages (negative: not seen, or not there).
struct Spot {
  int page[2];
  MGQA_DEV void look_up(const CacheAttnParams &p, const Piece &pc, int t, int gq) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      int kind;
      const int j = first_key(pc.rp, t, kShift, kind) + gq + 8 * i;
      page[i] = t < pc.t1 && !kind && wanted(pc.rp, 0, j) ? page_of(p, pc.b, j) : -2;
    }
  }
};

struct RowRule {
  float lse;  // of log2; +inf: the row has no weights to give
  float factor;
  int pos, lo;
};

template <typename K, int D>
__global__ void __launch_bounds__(kThreads, (K::ROWB == 512 ? 2 : 4))
cache_weights_kernel(const __grid_constant__ WeightParams wp) {
  using T = typename K::Query;
  const CacheAttnParams &p = wp.t.a;
  extern __shared__ __align__(16) unsigned char staged[];
  __shared__ RowRule rule[kChunkRows];
  __shared__ LocateScratch<kThreads> scratch;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, gq = lane >> 2, tq = lane & 3;
  if (warp == 1) touch_params(wp, lane);
  grid_dependency_wait();
  allow_dependents();
  Pieces pieces{};
  pieces.start<kThreads>(wp.t, scratch);
  Piece pc;
  while (pieces.next(p, pc)) {
    const RowPlan &rp = pc.rp;
    if (rp.np == 0) continue;
    for (int r0 = 0; r0 < p.R; r0 += wp.chunk) {
      const int rows = min(wp.chunk, p.R - r0), groups = (rows + 7) / 8;
      __syncthreads();  // the rows of an earlier chunk are no longer read
      for (int g8 = warp; g8 < groups; g8 += kWarps) {
        const int row = r0 + 8 * g8 + gq;
        const bool in = row < p.R;
        const int t = in ? row / p.n_rep : 0, h = pc.g * p.n_rep + (in ? row - t * p.n_rep : 0);
        const float f = K::stage(in ? static_cast<const T *>(p.q) + (int64_t)pc.b * p.qs[0] + (int64_t)h * p.qs[1] +
                                          (int64_t)t * p.qs[2]
                                    : static_cast<const T *>(nullptr),
                                 staged + g8 * K::STAGED, lane);
        if (tq == 0) {
          const float x = in ? __ldg(p.lse + ((int64_t)pc.b * p.Hq + h) * p.T + t) : -INFINITY;
          RowRule &rr = rule[8 * g8 + gq];
          rr.lse = x == -INFINITY ? INFINITY : x * kLog2e;
          rr.factor = f * p.scale_log2;
          rr.pos = in ? rp.n - p.T + t : -1;
          rr.lo = rr.pos - p.window + 1;
        }
      }
      __syncthreads();
      const int near = rp.n - p.T + r0 / p.n_rep, far = rp.n - p.T + (r0 + rows - 1) / p.n_rep - p.window + 1;
      K now, next;
      Spot spot;
      const auto fetch = [&](K &k, int t) {
        int kind;
        const int j0 = first_key(rp, t, kShift, kind) + gq;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          if (spot.page[i] == -1) report_error(p.err, MGQA_ERR_INVALID_ARG);
          if (spot.page[i] >= 0)
            k.load(i, static_cast<const char *>(p.k) + (int64_t)spot.page[i] * p.ks[0] + (int64_t)pc.g * p.ks[1] +
                          (int64_t)slot_in_page(p, j0 + 8 * i) * p.ks[2], tq);
          else
            k.clear(i);
        }
      };
      int t = pc.t0 + warp;
      spot.look_up(p, pc, t, gq);
      if (t < pc.t1) fetch(next, t);
      bool seen[2], seen_next[2] = {spot.page[0] >= 0, spot.page[1] >= 0};
      spot.look_up(p, pc, t + kWarps, gq);
      for (; t < pc.t1; t += kWarps) {
        now = next;
        seen[0] = seen_next[0];
        seen[1] = seen_next[1];
        if (t + kWarps < pc.t1) {
          fetch(next, t + kWarps);
          seen_next[0] = spot.page[0] >= 0;
          seen_next[1] = spot.page[1] >= 0;
          spot.look_up(p, pc, t + 2 * kWarps, gq);
        }
        int kind;
        const int k0 = first_key(rp, t, kShift, kind);
        const bool all = k0 + kKeys - 1 <= near && (k0 >= far || k0 + kKeys <= p.sinks);
        float w[2] = {0.f, 0.f};
        for (int g8 = 0; g8 < groups; ++g8) {
          float s[4];
          now.scores(staged + g8 * K::STAGED, lane, s);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const RowRule rr = rule[8 * g8 + 2 * tq + (e & 1)];
            const int j = k0 + gq + 8 * (e >> 1);
            const float x = fast_exp2(fmaf(s[e], rr.factor, -rr.lse));
            const bool see = all || (j <= rr.pos && (j >= rr.lo || j < p.sinks));
            w[e >> 1] += see ? x : 0.f;
          }
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          w[i] += __shfl_xor_sync(0xffffffffu, w[i], 1);
          w[i] += __shfl_xor_sync(0xffffffffu, w[i], 2);
          if (tq == i && seen[i]) {
            float *to = wp.weight + (int64_t)pc.b * wp.ws[0] + (int64_t)pc.g * wp.ws[1] + k0 + gq + 8 * i;
            *to = __ldcg(to) + w[i];
          }
        }
      }
    }
  }
}

template <typename K, int D>
mgqa_status launch_k(WeightParams wp, int sms, cudaStream_t s) {
  auto kern = cache_weights_kernel<K, D>;
  CacheAttnParams &p = wp.t.a;
  static std::atomic<uint64_t> attr{0};
  const mgqa_status st = ensure_smem_attr(kern, kChunkRows / 8 * K::STAGED, attr, "cache weights kernel");
  if (st != MGQA_OK) return st;
  p.RB = 1;
  p.block_rows = p.R;
  p.tile_shift = kShift;
  p.lead = 4;
  p.min_run = kWarps;
  wp.chunk = std::min(kChunkRows, (p.R + 7) / 8 * 8);
  const int64_t units = (int64_t)p.B * p.Hkv;
  const int grid = (int)std::max<int64_t>(1, std::min<int64_t>(4 * sms, units * (most_tiles(p) + p.lead)));
  const cudaError_t e =
      launch_pdl(kern, dim3(grid), dim3(kThreads), (size_t)(wp.chunk / 8) * K::STAGED, s, wp);
  if (e != cudaSuccess) return fail(MGQA_ERR_CUDA, "cache weights launch: %s", cudaGetErrorString(e));
  return MGQA_OK;
}
template <typename T>
mgqa_status launch_type(const WeightParams &wp, int D, bool q4, int sms, cudaStream_t s) {
  if (q4) return D == 64 ? launch_k<Q4Keys<T, 64>, 64>(wp, sms, s) : launch_k<Q4Keys<T, 128>, 128>(wp, sms, s);
  return D == 64 ? launch_k<Keys<T, 64>, 64>(wp, sms, s) : launch_k<Keys<T, 128>, 128>(wp, sms, s);
}

}  // namespace

mgqa_status launch_cache_weights(const mgqa_args &a, const mgqa_pages *pages, int32_t window, int32_t sinks, bool q4,
                                 float *weight, const int64_t *weight_stride, int32_t weight_slots, cudaStream_t s) {
  WeightParams wp{};
  cache_attn_params(a, pages, nullptr, window, sinks, wp.t.a);
  wp.t.a.cap = std::min(a.Lk, weight_slots);
  if (!q4)  // strides in bytes
    for (int t = 0; t < 3; ++t) wp.t.a.ks[t] *= a.dtype == MGQA_FP32 ? 4 : 2;
  wp.weight = weight;
  wp.ws[0] = weight_stride[0];
  wp.ws[1] = weight_stride[1];
  const int sms = device_sm_count();
  if (sms < 1) return fail(MGQA_ERR_CUDA, "cannot read the SM count of the current device");
  if (a.dtype == MGQA_BF16) return launch_type<__nv_bfloat16>(wp, a.D, q4, sms, s);
  if (a.dtype == MGQA_FP16) return launch_type<__half>(wp, a.D, q4, sms, s);
  return launch_type<float>(wp, a.D, q4, sms, s);
}

}  // namespace mgqa
