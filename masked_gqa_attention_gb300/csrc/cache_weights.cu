// What the last T cached tokens look at: the attention weights that they give to
// every slot of the cache, summed over the tokens and over the query heads of a KV
// head, and added to what earlier calls have found:
//   weight[b,g,j] += sum_{t, h in g} exp(scale <q[b,h,t], k[b,g,j]> - lse[b,h,t])
// over the slots j that token t sees (the rule of cache_q4.cu); lse comes from the
// attention call.
//
// Every visible key is read once, 2 D operations for each of R = T Hq / Hkv rows:
// up to some 64 rows the reads bound it, then the products. Keys are independent of
// one another, so every warp streams tiles of its own (cache_stream.cuh) and takes the
// keys as the first operand of m16n8k16 products with 8 rows of queries each, which
// the CTA has staged in shared memory in the order of their operand registers. fp32
// keys take the CUDA cores, a quad of lanes a key; keys in 4 bits the products of
// cache_q4.cuh. (32 requests of 16425 slots on average, 8 KV heads of 4 query heads,
// D = 128: bf16 175 us, 0.94 of the copy rate; fp32 334, 0.96; 4 bits 85, 0.64: 1.9
// instructions a cycle of four, warps that wait for their own last one. 32 tokens, so
// 128 rows, over two prompts of 28140: 54 us, four times the reads: chains of eight
// products, two warps a scheduler; fp32 571, some 200 of them the multiply-adds alone; 4
// bits 92, with fp32 queries 137. The forms for more than 8 rows that ask for three CTAs an
// SM spill 56 to 168 bytes a thread; with 128 rows staged two of the three fit for 4 bits,
// and of fp32 keys at D = 128 one of two, but the grid counts them all.)
//
// The tiles of all requests and KV heads are cut into equal runs (cache_sched.cuh);
// no sum crosses a warp but a quad's, so results repeat bit for bit.
#include <algorithm>

#include "cache_q4.cuh"
#include "cache_stream.cuh"

namespace mgqa {
namespace {

constexpr int kWarps = 4;
constexpr int kThreads = 32 * kWarps;
constexpr int kChunkRows = 128;  // query rows that are staged at a time

struct WeightParams {
  StreamParams s;
  float *weight;
  int64_t ws[2];  // request, KV head
  int32_t chunk;  // rows staged at a time: 8, or a multiple of 16
};

// The keys of a tile, as a lane holds them: block i has keys 8 i + gq. 16-bit (as the
// products take them: taken in 16-byte pieces, half of all instructions moved them) ...
template <typename T, int D>
struct Keys {
  using Query = T;
  static constexpr int KEYS = 32, N = D / 16;  // N: products
  static constexpr int ROWB = D * 2;
  static constexpr Order ORDER = kXor;
  static constexpr int STAGED = N * 256;  // bytes of 8 staged rows
  static constexpr int CTAS = 2, CTAS_ONE = D == 128 ? 2 : 3, STAGES = D == 128 ? 2 : 3;
  uint32_t k[2][N][4];

  MGQA_DEV void take(const unsigned char *tile, int lane) {
    const int row = lane & 15;
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
      for (int s = 0; s < N; ++s)
        ldmatrix_x4(k[m][s][0], k[m][s][1], k[m][s][2], k[m][s][3],
                    tile + (16 * m + row) * ROWB + ((2 * s + (lane >> 4)) ^ (row & 7)) * 16);
  }
  // Query row (null: zeros) of this lane's quad to its place of 8 staged rows; the
  // factor that its scores still need.
  static MGQA_DEV float stage(const T *row, unsigned char *to, int lane) {
    const uint32_t *src = reinterpret_cast<const uint32_t *>(row) + (lane & 3);
#pragma unroll
    for (int s = 0; s < N; s += 2)
      reinterpret_cast<uint4 *>(to)[s / 2 * 32 + lane] =
          row ? make_uint4(src[8 * s], src[8 * s + 4], src[8 * s + 8], src[8 * s + 12]) : make_uint4(0u, 0u, 0u, 0u);
    return 1.f;
  }
  // s[i][e]: block i with row 2 tq + e
  MGQA_DEV void scores(const unsigned char *staged, int lane, float (&s)[4][2], int = 8) const {
    float x[2][4];
#pragma unroll
    for (int c = 0; c < N; c += 2) {
      const uint4 q = reinterpret_cast<const uint4 *>(staged)[c / 2 * 32 + lane];
#pragma unroll
      for (int m = 0; m < 2; ++m) {
        const uint32_t(&a)[4] = k[m][c];
        if (c == 0) mma_16816_first<T>(x[m], a[0], a[1], a[2], a[3], q.x, q.y);
        else mma_16816<T>(x[m], a[0], a[1], a[2], a[3], q.x, q.y);
      }
#pragma unroll
      for (int m = 0; m < 2; ++m)
        mma_16816<T>(x[m], k[m][c + 1][0], k[m][c + 1][1], k[m][c + 1][2], k[m][c + 1][3], q.z, q.w);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      s[i][0] = x[i / 2][i % 2 * 2];
      s[i][1] = x[i / 2][i % 2 * 2 + 1];
    }
  }
};

// ... 32-bit, on the CUDA cores (two blocks) ...
template <int D>
struct Keys<float, D> {
  using Query = float;
  static constexpr int KEYS = 16, N = D / 16;
  static constexpr int ROWB = D * 4;
  static constexpr Order ORDER = kOddSwapped;
  static constexpr int STAGED = 8 * D * 4;
  static constexpr int CTAS = D == 128 ? 2 : 3, CTAS_ONE = CTAS, STAGES = 2;
  float4 k[2][N];

  MGQA_DEV void take(const unsigned char *tile, int lane) {
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int c = 0; c < N; ++c)
        k[i][c] = *reinterpret_cast<const float4 *>(tile + (8 * i + lane / 4) * ROWB + ((4 * c + lane % 4) ^ (lane & 4)) * 16);
  }
  static MGQA_DEV float stage(const float *row, unsigned char *to, int lane) {
#pragma unroll
    for (int c = 0; c < N; ++c)
      reinterpret_cast<float4 *>(to)[(lane >> 2) * (D / 4) + 4 * c + (lane & 3)] =
          row ? *(reinterpret_cast<const float4 *>(row) + 4 * c + (lane & 3)) : make_float4(0.f, 0.f, 0.f, 0.f);
    return 1.f;
  }
  // (rows: of the 8, how many there are)
  MGQA_DEV void scores(const unsigned char *staged, int lane, float (&s)[2][2], int rows = 8) const {
    const int tq = lane & 3;
    s[0][0] = s[0][1] = s[1][0] = s[1][1] = 0.f;
#pragma unroll
    for (int r = 0; r < 8; ++r) {
      if (r >= rows) break;
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
        s[0][r % 2] = x;
        s[1][r % 2] = y;
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
  static constexpr int KEYS = 32, N = F::CHUNKS;
  static constexpr int ROWB = F::REC;
  static constexpr Order ORDER = kAsIs;
  static constexpr int WORDS = 8 * F::KS;  // operand registers of a row, one term
  static constexpr int STAGED = (WORDS * (SPLIT ? 2 : 1) + 2) * 128;
  static constexpr int CTAS = 3, CTAS_ONE = 4, STAGES = 4;
  uint32_t w[N][4], par[2][4];
  float sc[4][4];

  MGQA_DEV void take(const unsigned char *tile, int lane) {
#pragma unroll
    for (int c = 0; c < N; ++c)
      ldmatrix_x4(w[c][0], w[c][1], w[c][2], w[c][3], tile + lane * F::REC + c * 16);
#pragma unroll
    for (int m = 0; m < 2; ++m)
      ldmatrix_x4(par[m][0], par[m][1], par[m][2], par[m][3], tile + (16 * m + (lane & 15)) * F::REC + F::CODES);
#pragma unroll
    for (int i = 0; i < 4; ++i) q4_four(tile + (8 * i + lane / 4) * F::REC + F::CODES, sc[i]);
  }
  static MGQA_DEV float stage(const T *row, unsigned char *to, int lane) {
    Q4Row<D, SPLIT> q;
    q.load(row, lane & 3);
    uint32_t *x = reinterpret_cast<uint32_t *>(to);
#pragma unroll
    for (int g = 0; g < 4; ++g)
#pragma unroll
      for (int i = 0; i < F::KS; ++i) {
        const int at = (g * F::KS + i) * 64 + 2 * lane;
        *reinterpret_cast<uint2 *>(x + at) = make_uint2(q.a[g][i][0], q.a[g][i][1]);
        if constexpr (SPLIT) *reinterpret_cast<uint2 *>(x + WORDS * 32 + at) = make_uint2(q.b[g][i][0], q.b[g][i][1]);
      }
    *reinterpret_cast<uint2 *>(x + (STAGED / 4 - 64) + 2 * lane) = make_uint2(q.sums[0], q.sums[1]);
    return q.down;
  }
  MGQA_DEV void scores(const unsigned char *staged, int lane, float (&s)[4][2], int = 8) const {
    const uint32_t *q = reinterpret_cast<const uint32_t *>(staged);
    const uint2 last = *reinterpret_cast<const uint2 *>(q + (STAGED / 4 - 64) + 2 * lane);
    const uint32_t sums[2] = {last.x, last.y};
    const auto term = [&](int t) {
      return [=](int g, int i) {
        return *reinterpret_cast<const uint2 *>(q + t * WORDS * 32 + (g * F::KS + i) * 64 + 2 * lane);
      };
    };
    Q4Scores<D, SPLIT> x[2];
#pragma unroll
    for (int m = 0; m < 2; ++m) x[m].least(par[m], sums);
#pragma unroll
    for (int c = 0; c < N; ++c)
#pragma unroll
      for (int m = 0; m < 2; ++m) {
        uint32_t u[2][4];
        q4_codes<SPLIT>(w[c][2 * m], u[0]);
        q4_codes<SPLIT>(w[c][2 * m + 1], u[1]);
        x[m].chunk(c, u, reinterpret_cast<const float(&)[2][4]>(sc[2 * m]), term(0), term(1));
      }
#pragma unroll
    for (int m = 0; m < 2; ++m) x[m].finish();
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      s[i][0] = x[i / 2].s[i % 2 * 2];
      s[i][1] = x[i / 2].s[i % 2 * 2 + 1];
    }
  }
};

struct RowRule {
  float lse;  // in units of log 2; +inf: the row has no weights to give
  float factor;
  int pos, pad;
};

template <typename K, int D>
struct Cfg {
  static constexpr int STAGES = K::STAGES;
  static constexpr int TILEB = K::KEYS * K::ROWB;
  static constexpr int ring = kWarps * STAGES * TILEB;
  struct Misc {
    RowRule rule[kChunkRows];
    LocateScratch<kThreads> scratch;
    int2 what[kWarps][STAGES];
    Feed feed[kWarps];
  };
  static constexpr int fixed = ring + (int)sizeof(Misc);  // the staged rows follow
};

// ONE: no more than 8 rows.
template <typename K, int D, bool ONE>
__global__ void __launch_bounds__(kThreads, ONE ? K::CTAS_ONE : K::CTAS)
cache_weights_kernel(const __grid_constant__ WeightParams wp) {
  using T = typename K::Query;
  using C = Cfg<K, D>;
  constexpr int STAGES = C::STAGES, NB = K::KEYS / 8;
  const CacheAttnParams &p = wp.s.t.a;
  extern __shared__ __align__(16) unsigned char smem[];
  auto &sm = *reinterpret_cast<typename C::Misc *>(smem + C::ring);
  unsigned char *staged = smem + C::fixed;
  const int tid = threadIdx.x, lane = lane_id(), warp = tid >> 5, gq = lane >> 2, tq = lane & 3;
  unsigned char *ring = smem + warp * (STAGES * C::TILEB);
  if (warp == 1) touch_params(wp, lane);
  grid_dependency_wait();
  allow_dependents();
  Pieces pieces{};
  pieces.start<kThreads>(wp.s.t, sm.scratch);

  const int passes = (p.R + wp.chunk - 1) / wp.chunk;
  Stream<K::KEYS, K::ROWB / 16, K::ORDER, false, kWarps> ahead(sm.feed[warp], passes);
  ahead.start(wp.s, pieces, warp, lane);
  int put = 0, st = 0;
  const auto start_one = [&] {
    if (ahead.live) {
      ahead.issue(wp.s, warp, lane, ring + put * C::TILEB, sm.what[warp] + put);
      put = put + 1 == STAGES ? 0 : put + 1;
    }
    cp_async_commit();
  };
  for (int s = 0; s < STAGES - 1; ++s) start_one();

  Piece pc;
  while (pieces.next(p, pc)) {
    const RowPlan &rp = pc.rp;
    for (int r0 = 0; r0 < p.R; r0 += wp.chunk) {
      // (eight rows, or pairs of them, with rows that give nothing behind the last one)
      const int rows = min(wp.chunk, p.R - r0), groups = ONE ? 1 : (rows + 15) / 16 * 2;
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
          sm.rule[8 * g8 + gq] = RowRule{x == -INFINITY ? INFINITY : x * kLog2e, f * p.scale_log2, in ? rp.n - p.T + t : -1, 0};
        }
      }
      __syncthreads();
      const int near = rp.n - p.T + r0 / p.n_rep, far = rp.n - p.T + (r0 + rows - 1) / p.n_rep - p.window + 1;
      for (int t = pc.t0 + warp; t < pc.t1; t += kWarps) {
        start_one();
        cp_async_wait<STAGES - 1>();
        __syncwarp();
        const int k0 = sm.what[warp][st].x;
        const uint32_t okw = (uint32_t)sm.what[warp][st].y;
        // lane (gq, tq) adds to the weight of key 8 tq + gq
        const int mine = 8 * tq + gq;
        const bool seen = tq < NB && (okw >> mine & 1u);
        float *to = wp.weight + (int64_t)pc.b * wp.ws[0] + (int64_t)pc.g * wp.ws[1] + k0 + mine;
        const float old = seen ? __ldcg(to) : 0.f;
        K keys;
        keys.take(ring + st * C::TILEB, lane);
        const bool all = k0 + K::KEYS - 1 <= near && (k0 >= far || k0 + K::KEYS <= p.sinks);
        float w[NB] = {};
        const auto add = [&](int g8, float (&s)[NB][2]) {  // the weights of 8 rows
          const int4 ra = *reinterpret_cast<const int4 *>(&sm.rule[8 * g8 + 2 * tq]);
          const int4 rb = *reinterpret_cast<const int4 *>(&sm.rule[8 * g8 + 2 * tq + 1]);
          const float lse[2] = {__int_as_float(ra.x), __int_as_float(rb.x)}, f[2] = {__int_as_float(ra.y), __int_as_float(rb.y)};
#pragma unroll
          for (int i = 0; i < NB; ++i)
#pragma unroll
            for (int e = 0; e < 2; ++e) s[i][e] = fast_exp2(fmaf(s[i][e], f[e], -lse[e]));
          if (!all) {
            const int pos[2] = {ra.z, rb.z};
#pragma unroll
            for (int i = 0; i < NB; ++i)
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                const int j = k0 + 8 * i + gq;
                const bool see = j <= pos[e] && (j > pos[e] - p.window || j < p.sinks);
                s[i][e] = see ? s[i][e] : 0.f;
              }
          }
#pragma unroll
          for (int i = 0; i < NB; ++i) w[i] += s[i][0] + s[i][1];
        };
        if constexpr (ONE) {
          float s[NB][2];
          keys.scores(staged, lane, s, rows);
          add(0, s);
        } else {
          for (int g8 = 0; g8 < groups; g8 += 2) {  // (two at a time: one's products are a chain)
            float s[NB][2], z[NB][2];
            keys.scores(staged + g8 * K::STAGED, lane, s);
            keys.scores(staged + (g8 + 1) * K::STAGED, lane, z);
            add(g8, s);
            add(g8 + 1, z);
          }
        }
        float sum = 0.f;
#pragma unroll
        for (int i = 0; i < NB; ++i) {
          w[i] += __shfl_xor_sync(0xffffffffu, w[i], 1);
          w[i] += __shfl_xor_sync(0xffffffffu, w[i], 2);
          sum = tq == i ? w[i] : sum;
        }
        if (seen) *to = old + sum;
        __syncwarp();  // the stage has been read
        st = st + 1 == STAGES ? 0 : st + 1;
      }
    }
  }
}

template <typename K, int D, bool ONE>
mgqa_status launch_k(WeightParams wp, int page_size, int sms, cudaStream_t s) {
  using C = Cfg<K, D>;
  auto kern = cache_weights_kernel<K, D, ONE>;
  CacheAttnParams &p = wp.s.t.a;
  static std::atomic<uint64_t> attr{0};
  const mgqa_status st = ensure_smem_attr(kern, C::fixed + kChunkRows / 8 * K::STAGED, attr, "cache weights kernel");
  if (st != MGQA_OK) return st;
  if (!set_steps(wp.s, p.ks, nullptr, K::ROWB, page_size))
    return fail(MGQA_ERR_UNSUPPORTED, "strides of the cache past 2^36 bytes");
  p.RB = 1;
  p.block_rows = p.R;
  p.tile_shift = K::KEYS == 32 ? 5 : 4;
  p.lead = 4;
  p.min_run = kWarps;
  wp.chunk = ONE ? 8 : std::min(kChunkRows, (p.R + 15) / 16 * 16);
  const int64_t units = (int64_t)p.B * p.Hkv;
  const int grid = (int)std::max<int64_t>(1, std::min<int64_t>((ONE ? K::CTAS_ONE : K::CTAS) * sms, units * (most_tiles(p) + p.lead)));
  const cudaError_t e = launch_pdl(kern, dim3(grid), dim3(kThreads), (size_t)C::fixed + (wp.chunk / 8) * K::STAGED, s, wp);
  if (e != cudaSuccess) return fail(MGQA_ERR_CUDA, "cache weights launch: %s", cudaGetErrorString(e));
  return MGQA_OK;
}
template <typename K, int D>
mgqa_status launch_k(const WeightParams &wp, int page_size, int sms, cudaStream_t s) {
  return wp.s.t.a.R <= 8 ? launch_k<K, D, true>(wp, page_size, sms, s) : launch_k<K, D, false>(wp, page_size, sms, s);
}
template <typename T>
mgqa_status launch_type(const WeightParams &wp, int D, bool q4, int page_size, int sms, cudaStream_t s) {
  if (q4)
    return D == 64 ? launch_k<Q4Keys<T, 64>, 64>(wp, page_size, sms, s) : launch_k<Q4Keys<T, 128>, 128>(wp, page_size, sms, s);
  return D == 64 ? launch_k<Keys<T, 64>, 64>(wp, page_size, sms, s) : launch_k<Keys<T, 128>, 128>(wp, page_size, sms, s);
}

}  // namespace

mgqa_status launch_cache_weights(const mgqa_args &a, const mgqa_pages *pages, int32_t window, int32_t sinks, bool q4,
                                 float *weight, const int64_t *weight_stride, int32_t weight_slots, cudaStream_t s) {
  WeightParams wp{};
  CacheAttnParams &p = wp.s.t.a;
  cache_attn_params(a, pages, nullptr, window, sinks, p);
  p.cap = std::min(a.Lk, weight_slots);
  if (!q4)  // strides in bytes
    for (int t = 0; t < 3; ++t) p.ks[t] *= a.dtype == MGQA_FP32 ? 4 : 2;
  wp.weight = weight;
  wp.ws[0] = weight_stride[0];
  wp.ws[1] = weight_stride[1];
  const int sms = device_sm_count(), page_size = pages ? pages->page_size : 0;
  if (sms < 1) return fail(MGQA_ERR_CUDA, "cannot read the SM count of the current device");
  if (a.dtype == MGQA_BF16) return launch_type<__nv_bfloat16>(wp, a.D, q4, page_size, sms, s);
  if (a.dtype == MGQA_FP16) return launch_type<__half>(wp, a.D, q4, page_size, sms, s);
  return launch_type<float>(wp, a.D, q4, page_size, sms, s);
}

}  // namespace mgqa
