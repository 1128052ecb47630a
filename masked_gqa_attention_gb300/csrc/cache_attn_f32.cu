// The fp32 cache attention: the formulas of cache_attn.cu on the CUDA cores
// (single-precision accuracy rules the tensor cores out), with the tiles, the two
// ways to cut the work and the producer warps of cache_attn_tma.cu.
//
// A key is 8 D bytes and 4 R D operations: up to R = 4 the reads bound it (64 rows
// of up to 32768 slots, window 4096, R = 4: 323 us, 90 % of the copy rate; R = 8:
// 640), beyond that the CUDA cores. Two forms:
//   16 rows or fewer: a thread has 4 rows and one key of the scores (a quarter,
//     half or all of the head dim), then 4 rows and 4 features of the values
//     (every 8th, 4th or 2nd key), so each K and V element is read from shared
//     memory once per 4 rows; two block barriers a tile.
//   32, 48 or 64 rows: the register tiles of simt_fp32.cuh.
#include <algorithm>
#include <cmath>

#include "cache_producer.cuh"
#include "simt_fp32.cuh"

namespace mgqa {
namespace {

constexpr int kConsumers = 256;
constexpr int kThreads = kConsumers + 64;

template <int D>
struct Ring {
  static constexpr int KB = D / 32;
  static constexpr int TILEB = KB * simt::kBox;  // bytes of a K (or V) tile
};

// ---- 16 rows or fewer: RG groups of 4 rows ------------------------------------------

template <int D, int RG>
struct FewCfg {
  static constexpr int ROWS = 4 * RG;
  static constexpr int DS = 4 / RG;                 // parts of the head dim in the scores
  static constexpr int FC = D / 4;                  // 16-byte columns of a row
  static constexpr int KS = kConsumers / FC / RG;   // parts of the keys in the values
  static constexpr int STAGES = 196608 / (2 * Ring<D>::TILEB) < 4 ? 196608 / (2 * Ring<D>::TILEB) : 4;
  static constexpr int ring = STAGES * 2 * Ring<D>::TILEB;
  static constexpr int OP = D + 4;
  static constexpr int SP = kTile + 4;
  struct Work {
    float s[DS][ROWS][SP];               // scores, by parts of the head dim
    float p[kTile][RG][4][2];            // weights, each twice
  };
  struct Misc {
    float q[ROWS][D];
    union {
      Work w;
      float o[KS > 1 ? KS - 1 : 1][ROWS][D];  // after the last tile: the other parts' results
    };
    float f[ROWS];
    float2 ml[ROWS];
    Drafts<32> drafts;
    LocateScratch<kThreads> scratch;
    uint2 ok[STAGES];
    uint64_t full[STAGES], empty[STAGES];
    int maxdepth;
  };
  static constexpr int threads = kThreads;
  static constexpr int smem = ring + (int)sizeof(Misc) + 1024;
  static_assert(smem <= 227 * 1024, "shared memory");
};

// ---- 32, 48 or 64 rows ---------------------------------------------------------------------

template <int D, int RPG>
struct ManyCfg {
  static constexpr int ROWS = 8 * RPG;
  static constexpr int STAGES = 131072 / (2 * Ring<D>::TILEB);
  static constexpr int ring = STAGES * 2 * Ring<D>::TILEB;
  static constexpr int QP = D + 4, OP = D + 4;
  // a third warpgroup with the producers gives its registers to the two others
  // (104 + 2 x 200 = 3 x 168, the launch's)
  static constexpr int threads = kConsumers + 128;
  struct Misc {
    float q[ROWS][QP];
    simt::Shared<ROWS, D> sh;
    float2 ml[ROWS];
    Drafts<kMaxDrafts> drafts;
    LocateScratch<threads> scratch;
    uint2 ok[STAGES];
    uint64_t full[STAGES], empty[STAGES];
    int maxdepth;
  };
  static constexpr int smem = ring + (int)sizeof(Misc) + 1024;
  static_assert(smem <= 227 * 1024, "shared memory");
};

// What both kernels do at a piece's start: the query rows (in shared memory, row
// pitch QP) and, when its masks need them, the drafts.
template <int D, int ROWS, int QP, int MAXT>
MGQA_DEV bool begin_piece(const CacheAttnParams &p, const Piece &pc, int row0, float *q, Drafts<MAXT> &drafts,
                          int &maxdepth, int &staged) {
  const int tid = threadIdx.x;
  named_sync(1, kConsumers);  // the previous piece's readers are done
#pragma unroll
  for (int u0 = 0; u0 < ROWS * (D / 4); u0 += kConsumers) {
    const int u = u0 + tid;
    if (u < ROWS * (D / 4)) {
      const int r = u / (D / 4), d = (u % (D / 4)) * 4, row = row0 + r, t = row / p.n_rep;
      float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
      if (row < p.R)
        x = *reinterpret_cast<const float4 *>(static_cast<const float *>(p.q) + (int64_t)pc.b * p.qs[0] +
                                              (int64_t)(pc.g * p.n_rep + row - t * p.n_rep) * p.qs[1] +
                                              (int64_t)t * p.qs[2] + d);
      *reinterpret_cast<float4 *>(q + r * QP + d) = x;
    }
  }
  const bool need = p.tree && (p.window != kNoWindow || pc.t1 > pc.rp.np);
  if (need && staged != pc.b) {
    if (tid == 0) maxdepth = 0;
    stage_drafts(p, drafts, pc.b, pc.rp.live, tid, kConsumers);
    named_sync(1, kConsumers);
    if (tid < pc.rp.live && drafts.depth[tid]) atomicMax(&maxdepth, drafts.depth[tid]);
    staged = pc.b;
  }
  named_sync(1, kConsumers);
  return need;
}

template <int MAXT>
MGQA_DEV RowSight sight_of(const CacheAttnParams &p, const Piece &pc, int row, bool need, const Drafts<MAXT> &drafts) {
  RowSight s;
  s.t = row / p.n_rep;
  s.ok = row < p.R && (!p.tree || s.t < pc.rp.live);
  const int pt = p.tree ? pc.rp.n + (need && s.ok ? drafts.depth[s.t] : 0) : pc.rp.n - 1;
  s.lo = pt - p.window + 1;
  return s;
}

template <int D, int RG>
__global__ void __launch_bounds__(kThreads, 1)
cache_attn_f32_few_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                          const __grid_constant__ CUtensorMap tm_kn, const __grid_constant__ CUtensorMap tm_vn,
                          const __grid_constant__ TmaParams tp) {
  using C = FewCfg<D, RG>;
  constexpr int ROWS = C::ROWS, STAGES = C::STAGES, DS = C::DS, FC = C::FC, KS = C::KS, TILEB = Ring<D>::TILEB;
  const CacheAttnParams &p = tp.a;
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  unsigned char *ring = reinterpret_cast<unsigned char *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
  auto &sm = *reinterpret_cast<typename C::Misc *>(ring + C::ring);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (tid == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(sm.full + s, full_count(tp));
      mbar_init(sm.empty + s, kConsumers / 32);
    }
    fence_mbarrier_init();
  }
  if (warp == 1) touch_params(tp, lane);
  grid_dependency_wait();
  allow_dependents();
  Pieces pieces{};
  pieces.start<kThreads>(tp, sm.scratch);
  if (warp >= kConsumers / 32) {
    const int of_v = warp - kConsumers / 32;
    produce_tiles<Ring<D>::KB, 32, STAGES>(tp, pieces, of_v, of_v ? &tm_v : &tm_k, of_v ? &tm_vn : &tm_kn, ring,
                                           sm.ok, sm.full, sm.empty);
  } else {
    if (pieces.idle() && tid < ROWS) sm.ml[tid] = make_float2(-INFINITY, 0.f);
    bool ok = true;
    int it = 0, staged = -1;
    Piece pc;
    while (pieces.next(p, pc)) {
      const RowPlan &rp = pc.rp;
      const PieceOut po = out_of(p, pc, blockIdx.x);
      const bool need = begin_piece<D, ROWS, D>(p, pc, po.row0, &sm.q[0][0], sm.drafts, sm.maxdepth, staged);
      // scores: key `key`, rows 4 sg .. + 3, part sd of the head dim
      const int key = tid & 63, sg = (tid >> 6) % RG, sd = (tid >> 6) / RG;
      // softmax: this warp's rows warp, warp + 8; lane has keys lane, lane + 32
      constexpr int RPW = (ROWS + 7) / 8;
      RowSight sight[RPW];
      float m[RPW], l[RPW];
#pragma unroll
      for (int i = 0; i < RPW; ++i) {
        sight[i] = sight_of(p, pc, po.row0 + warp + 8 * i, need, sm.drafts);
        m[i] = -INFINITY;
        l[i] = 0.f;
      }
      // values: features 4 fc .. + 3 of rows 4 vg .. + 3, keys vk, vk + KS, ...
      const int fc = tid % FC, vg = tid / FC % RG, vk = tid / FC / RG;
      uint64_t o[4][2];
#pragma unroll
      for (int r = 0; r < 4; ++r) o[r][0] = o[r][1] = 0ull;

      for (int t = pc.t0; t < pc.t1; ++t, ++it) {
        const int st = it % STAGES;
        // (every thread has the same outcome: the barriers below are taken by all)
        if (ok) ok = __all_sync(0xffffffffu, mbar_wait(sm.full + st, (it / STAGES) & 1, p.err));
        const unsigned char *kt = ring + st * 2 * TILEB, *vt = kt + TILEB;
        const uint2 okw = sm.ok[st];
        {
          uint64_t acc[4] = {0ull, 0ull, 0ull, 0ull};
          constexpr int CH = FC / DS;
#pragma unroll 4
          for (int j = 0; j < CH; ++j) {
            const int c = sd * CH + j;
            uint64_t k0, k1;
            simt::lds_pairs(k0, k1, kt + (c >> 3) * simt::kBox + key * 128 + (((c & 7) ^ (key & 7)) << 4));
#pragma unroll
            for (int r = 0; r < 4; ++r) {
              uint64_t q0, q1;
              simt::lds_pairs(q0, q1, &sm.q[sg * 4 + r][c * 4]);
              acc[r] = tc::fma2(q0, k0, acc[r]);
              acc[r] = tc::fma2(q1, k1, acc[r]);
            }
          }
#pragma unroll
          for (int r = 0; r < 4; ++r) sm.w.s[sd][sg * 4 + r][key] = simt::pair_sum(acc[r]);
        }
        named_sync(1, kConsumers);
        int kind;
        const int k0 = first_key(rp, t, 6, kind);
#pragma unroll
        for (int i = 0; i < RPW; ++i) {
          const int row = warp + 8 * i;
          if (row < ROWS) {
            float x[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const int c = lane + 32 * e;
              float v = 0.f;
#pragma unroll
              for (int d = 0; d < DS; ++d) v += sm.w.s[d][row][c];
              const bool see = ((e ? okw.y : okw.x) >> lane & 1u) &&
                               (kind ? sees_draft(p, sm.drafts, sight[i], rp.n, k0 + c) : sees_cached(p, sight[i], k0 + c));
              x[e] = see ? v * p.scale_log2 : -INFINITY;
            }
            float mx = fmaxf(m[i], fmaxf(x[0], x[1]));
#pragma unroll
            for (int off = 16; off > 0; off >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, off));
            const float mb = mx == -INFINITY ? 0.f : mx;
            const float f = exp2f(m[i] - mb), w0 = exp2f(x[0] - mb), w1 = exp2f(x[1] - mb);
            m[i] = mx;
            l[i] = l[i] * f + w0 + w1;
            *reinterpret_cast<float2 *>(sm.w.p[lane][row / 4][row % 4]) = make_float2(w0, w0);
            *reinterpret_cast<float2 *>(sm.w.p[lane + 32][row / 4][row % 4]) = make_float2(w1, w1);
            if (lane == 0) sm.f[row] = f;
          }
        }
        named_sync(1, kConsumers);
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const float f = sm.f[vg * 4 + r];
          o[r][0] = simt::mul2(o[r][0], f);
          o[r][1] = simt::mul2(o[r][1], f);
        }
        const bool clean = (okw.x & okw.y) == 0xffffffffu;
#pragma unroll 4
        for (int j = 0; j < kTile / KS; ++j) {
          const int k = vk + j * KS;
          // (a key that does not count may hold anything: left out)
          if (!clean && !(((k < 32 ? okw.x : okw.y) >> (k & 31)) & 1u)) continue;
          uint64_t v0, v1, w[4];
          simt::lds_pairs(v0, v1, vt + (fc >> 3) * simt::kBox + k * 128 + (((fc & 7) ^ (k & 7)) << 4));
          simt::lds_pairs(w[0], w[1], sm.w.p[k][vg][0]);
          simt::lds_pairs(w[2], w[3], sm.w.p[k][vg][2]);
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            o[r][0] = tc::fma2(w[r], v0, o[r][0]);
            o[r][1] = tc::fma2(w[r], v1, o[r][1]);
          }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(sm.empty + st);
      }
      // ---- the rows' (m, l), and the parts of the keys together
#pragma unroll
      for (int i = 0; i < RPW; ++i) {
        float ls = l[i];
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) ls += __shfl_xor_sync(0xffffffffu, ls, off);
        const int row = warp + 8 * i;
        const bool none = !ok || !sight[i].ok || m[i] == -INFINITY;
        if (lane == 0 && row < ROWS) sm.ml[row] = none ? make_float2(-INFINITY, 0.f) : make_float2(m[i], ls);
      }
      named_sync(1, kConsumers);  // (also: the weights have been read)
      float x[4][4];
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        tc::upk2(o[r][0], x[r][0], x[r][1]);
        tc::upk2(o[r][1], x[r][2], x[r][3]);
        if (vk > 0)
          *reinterpret_cast<float4 *>(&sm.o[vk - 1][vg * 4 + r][fc * 4]) = make_float4(x[r][0], x[r][1], x[r][2], x[r][3]);
      }
      named_sync(1, kConsumers);
      if (vk == 0)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const int row = vg * 4 + r;
          const float2 ml = sm.ml[row];
#pragma unroll
          for (int k = 1; k < KS; ++k) {
            const float4 y = *reinterpret_cast<const float4 *>(&sm.o[k - 1][row][fc * 4]);
            x[r][0] += y.x;
            x[r][1] += y.y;
            x[r][2] += y.z;
            x[r][3] += y.w;
          }
          if (ml.x == -INFINITY) x[r][0] = x[r][1] = x[r][2] = x[r][3] = 0.f;
          if (pieces.S)
            *reinterpret_cast<float4 *>(reinterpret_cast<float *>(ring) + row * C::OP + fc * 4) =
                make_float4(x[r][0], x[r][1], x[r][2], x[r][3]);
          else if (row < po.rows)
            RowOut<float, D, ROWS>(p, po, row, ml.x, ml.y, fc == 0).put(fc * 4, x[r]);
        }
    }
  }
  if (pieces.S) join_cluster<float, D, ROWS, C::OP, kConsumers>(p, pieces, sm.ml, reinterpret_cast<const float *>(ring));
}

template <int D, int RPG>
__global__ void __launch_bounds__(kConsumers + 128, 1)
cache_attn_f32_many_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                           const __grid_constant__ CUtensorMap tm_kn, const __grid_constant__ CUtensorMap tm_vn,
                           const __grid_constant__ TmaParams tp) {
  using C = ManyCfg<D, RPG>;
  constexpr int ROWS = C::ROWS, STAGES = C::STAGES, TILEB = Ring<D>::TILEB;
  const CacheAttnParams &p = tp.a;
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  unsigned char *ring = reinterpret_cast<unsigned char *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
  auto &sm = *reinterpret_cast<typename C::Misc *>(ring + C::ring);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (tid == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(sm.full + s, full_count(tp));
      mbar_init(sm.empty + s, kConsumers / 32);
    }
    fence_mbarrier_init();
  }
  if (warp == 1) touch_params(tp, lane);
  grid_dependency_wait();
  allow_dependents();
  Pieces pieces{};
  pieces.start<C::threads>(tp, sm.scratch);
  if (warp >= kConsumers / 32) {
    tc::regs_dec<104>();
    const int of_v = warp - kConsumers / 32;
    if (of_v < 2)
      produce_tiles<Ring<D>::KB, 32, STAGES>(tp, pieces, of_v, of_v ? &tm_v : &tm_k, of_v ? &tm_vn : &tm_kn, ring,
                                             sm.ok, sm.full, sm.empty);
  } else {
    tc::regs_inc<200>();
    if (pieces.idle() && tid < ROWS) sm.ml[tid] = make_float2(-INFINITY, 0.f);
    const simt::Place at(tid);
    bool ok = true;
    int it = 0, staged = -1;
    Piece pc;
    while (pieces.next(p, pc)) {
      const RowPlan &rp = pc.rp;
      const PieceOut po = out_of(p, pc, blockIdx.x);
      const bool need = begin_piece<D, ROWS, C::QP>(p, pc, po.row0, &sm.q[0][0], sm.drafts, sm.maxdepth, staged);
      RowSight sight[RPG / 2];
      float m[RPG / 2], l[RPG / 2];
      uint64_t o[RPG][D / 64][2];
#pragma unroll
      for (int a = 0; a < RPG / 2; ++a) {
        sight[a] = sight_of(p, pc, po.row0 + at.own<RPG>(a), need, sm.drafts);
        m[a] = -INFINITY;
        l[a] = 0.f;
      }
#pragma unroll
      for (int a = 0; a < RPG; ++a)
#pragma unroll
        for (int c = 0; c < D / 64; ++c) o[a][c][0] = o[a][c][1] = 0ull;
      const int lo_all = rp.n + (p.tree ? (need ? sm.maxdepth : 0) : -1) - p.window + 1;
      for (int t = pc.t0; t < pc.t1; ++t, ++it) {
        const int st = it % STAGES;
        if (ok) ok = __all_sync(0xffffffffu, mbar_wait(sm.full + st, (it / STAGES) & 1, p.err));
        const unsigned char *kt = ring + st * 2 * TILEB;
        const uint2 okw = sm.ok[st];
        int kind;
        const int k0 = first_key(rp, t, 6, kind);
        const bool full = !kind && (okw.x & okw.y) == 0xffffffffu &&
                          (k0 >= lo_all || k0 + kTile <= min(p.sinks, rp.s_end));
        simt::tile<D, RPG, C::QP>(ok, it & 1, &sm.q[0][0], kt, kt + TILEB, sm.sh, o, m, l, at, okw.x, okw.y,
                                  [&](int a, int col, float s) {
                                    const bool see =
                                        full || (((col < 32 ? okw.x : okw.y) >> (col & 31) & 1u) &&
                                                 (kind ? sees_draft(p, sm.drafts, sight[a], rp.n, k0 + col)
                                                       : sees_cached(p, sight[a], k0 + col)));
                                    return see ? s * p.scale_log2 : -INFINITY;
                                  });
        __syncwarp();
        if (lane == 0) mbar_arrive(sm.empty + st);
      }
      float x[RPG / 2][D / 64][4];
      simt::finish<D, RPG>(sm.sh, o, l, x, at);  // (its barriers: every tile has been read, the ring takes the result)
#pragma unroll
      for (int a = 0; a < RPG / 2; ++a) {
        const int r = at.own<RPG>(a);
        const bool none = !ok || !sight[a].ok || m[a] == -INFINITY;
        const float2 ml = none ? make_float2(-INFINITY, 0.f) : make_float2(m[a], l[a]);
        const RowOut<float, D, ROWS> dst(p, po, r < po.rows ? r : 0, ml.x, ml.y,
                                         !pieces.S && at.tx == 0 && r < po.rows);
        if (pieces.S && at.tx == 0) sm.ml[r] = ml;
#pragma unroll
        for (int c = 0; c < D / 64; ++c) {
          if (none) x[a][c][0] = x[a][c][1] = x[a][c][2] = x[a][c][3] = 0.f;
          if (pieces.S)
            *reinterpret_cast<float4 *>(reinterpret_cast<float *>(ring) + r * C::OP + at.tx * 4 + 64 * c) =
                make_float4(x[a][c][0], x[a][c][1], x[a][c][2], x[a][c][3]);
          else if (r < po.rows)
            dst.put(at.tx * 4 + 64 * c, x[a][c]);
        }
      }
    }
  }
  if (pieces.S) join_cluster<float, D, ROWS, C::OP, kConsumers>(p, pieces, sm.ml, reinterpret_cast<const float *>(ring));
}

template <int D, typename C, typename Kern>
mgqa_status launch_t(Kern kern, std::atomic<uint64_t> &attr, const CUtensorMap (&maps)[4], TmaParams tp, int lead,
                     const CacheAttnLaunch &how, cudaStream_t s) {
  mgqa_status st = ensure_cluster_attr(kern, C::smem, attr, "fp32 cache attention kernel");
  if (st != MGQA_OK) return st;
  CacheAttnParams &p = tp.a;
  p.block_rows = C::ROWS;
  p.RB = (p.R + C::ROWS - 1) / C::ROWS;
  p.tile_shift = 6;
  const int64_t units = (int64_t)p.B * p.Hkv * p.RB, tiles = most_tiles(p);
  tp.cluster = cluster_size(p, D * 4, how.sms);
  if (tp.cluster) {
    const cudaError_t e = launch_pdl_cluster(kern, dim3((unsigned)(units * tp.cluster)), dim3(C::threads), C::smem, s,
                                             tp.cluster, maps[0], maps[1], maps[2], maps[3], tp);
    if (e != cudaSuccess) return fail(MGQA_ERR_CUDA, "fp32 cache attention launch: %s", cudaGetErrorString(e));
    return MGQA_OK;
  }
  p.lead = lead;
  p.min_run = 4;
  const int grid = (int)std::max<int64_t>(1, std::min<int64_t>(std::min(how.sms, kCacheAttnMaxCtas), units * (tiles + lead)));
  set_partials(p, how.workspace, grid, C::ROWS, D);
  const cudaError_t e = launch_pdl(kern, dim3(grid), dim3(C::threads), C::smem, s, maps[0], maps[1], maps[2], maps[3], tp);
  if (e != cudaSuccess) return fail(MGQA_ERR_CUDA, "fp32 cache attention launch: %s", cudaGetErrorString(e));
  return launch_cache_merge(p, MGQA_FP32, D, C::ROWS, grid, s);
}

template <int D, int RG>
mgqa_status launch_few(const CUtensorMap (&maps)[4], const TmaParams &tp, const CacheAttnLaunch &how, cudaStream_t s) {
  static std::atomic<uint64_t> attr{0};
  return launch_t<D, FewCfg<D, RG>>(cache_attn_f32_few_kernel<D, RG>, attr, maps, tp, 3, how, s);
}
template <int D, int RPG>
mgqa_status launch_many(const CUtensorMap (&maps)[4], const TmaParams &tp, const CacheAttnLaunch &how, cudaStream_t s) {
  static std::atomic<uint64_t> attr{0};
  return launch_t<D, ManyCfg<D, RPG>>(cache_attn_f32_many_kernel<D, RPG>, attr, maps, tp, 1, how, s);
}

template <int D>
mgqa_status launch_d(const CUtensorMap (&maps)[4], const TmaParams &tp, const CacheAttnLaunch &how, cudaStream_t s) {
  // the smallest block that holds the rows, or a smaller one of its kind on short
  // calls (one row of 16 heads over 2, window 1024, D = 64: 7.6 us in blocks of 4
  // rows, 9.0 in one of 8; 8 drafts over 4096 slots 11.5 in blocks of 32, 15.7 in
  // one of 64, 20 in blocks of 8)
  const CacheAttnParams &p = tp.a;
  int rows = p.R <= 4 ? 4 : p.R <= 8 ? 8 : 16;
  if (p.R > 16) {
    // more rows: the blocks that cost least together; a tile of one costs as its rows
    // and 6 more (32 rows 343, 64 rows 635 us for the same tiles; 16 trees of 24
    // drafts and 4 heads, 96 rows: 1270 us in two blocks of 64, 946 in two of 48)
    auto cost = [&](int r) { return (int64_t)((p.R + r - 1) / r) * (r + 6); };
    rows = cost(48) < cost(64) ? 48 : 64;
    if (cost(32) < cost(rows)) rows = 32;
  }
  if (p.T <= 32 && rows != 48) rows = short_block(p, D * 4, how.sms, rows, rows > 16 ? 32 : 4);
  if (rows == 4) return launch_few<D, 1>(maps, tp, how, s);
  if (rows == 8) return launch_few<D, 2>(maps, tp, how, s);
  if (rows == 16) return launch_few<D, 4>(maps, tp, how, s);
  if (rows == 32) return launch_many<D, 4>(maps, tp, how, s);
  if (rows == 48) return launch_many<D, 6>(maps, tp, how, s);
  return launch_many<D, 8>(maps, tp, how, s);
}

}  // namespace

mgqa_status launch_cache_attn_f32(const CacheAttnParams &p, int D, const CacheAttnLaunch &how, cudaStream_t s) {
  TmaParams tp{};
  tp.a = p;
  CUtensorMap maps[4];
  if (!cache_attn_maps(p, MGQA_FP32, D, kTile, maps, tp.box_rows))
    return fail(MGQA_ERR_CUDA, "cuTensorMapEncodeTiled failed for the cache");
  return D == 64 ? launch_d<64>(maps, tp, how, s) : launch_d<128>(maps, tp, how, s);
}

}  // namespace mgqa
