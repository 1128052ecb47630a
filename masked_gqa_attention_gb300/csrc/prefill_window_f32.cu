// Windowed prefill in fp32 on the CUDA cores.
//
// A window of W keys costs 4 W D operations per query and head against 4 D bytes
// of keys shared by 64 queries, so the fp32 rate bounds it. CTA = 64 query rows
// of one head; a producer warp fetches the 64-key tiles that the window and the
// sinks reach (TMA boxes, two stages at D = 128), 256 threads run the register
// tiles of simt_fp32.cuh; partial tiles take their mask words from shared memory.
// Tiles behind a request's kv_len are fetched and masked like any other.
// The last rows, which have the most keys under a causal limit, start first
// (4096 queries x 16 heads, window 4096: 1854 us, in rising order 2153). (The
// unwindowed fp32 prefill keeps its kernel of four threads per row, which took
// 5.2 ms of that.)
#include <algorithm>
#include <cmath>

#include "cache_sched.cuh"
#include "simt_fp32.cuh"

namespace mgqa {
namespace {

constexpr int kConsumers = 256;
constexpr int kThreads = kConsumers + 128;  // (a warpgroup for the producer, whose registers the others get)
constexpr int kRPG = 8, kRows = 8 * kRPG;

struct WinParams {
  const float *q;
  float *out;
  int64_t qs[3], os[3];
  MaskView mask;
  float scale_log2;
  float *lse;
  int32_t *err;
  int Hq, Lq, Lk, n_rep;
};

template <int D>
struct WinCfg {
  static constexpr int KB = D / 32;
  static constexpr int TILEB = KB * simt::kBox;
  static constexpr int STAGES = 131072 / (2 * TILEB);
  static constexpr int ring = STAGES * 2 * TILEB;
  static constexpr int QP = D + 4;
  struct Misc {
    float q[kRows][QP];
    simt::Shared<kRows, D> sh;
    uint32_t mask[2][kRows][2];  // of alternating partial tiles
    uint64_t full[STAGES], empty[STAGES];
  };
  static constexpr int smem = ring + (int)sizeof(Misc) + 1024;
  static_assert(smem <= 227 * 1024, "shared memory");
};

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
prefill_window_f32_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                          const __grid_constant__ WinParams p) {
  using C = WinCfg<D>;
  constexpr int STAGES = C::STAGES, TILEB = C::TILEB;
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  unsigned char *ring = reinterpret_cast<unsigned char *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
  auto &sm = *reinterpret_cast<typename C::Misc *>(ring + C::ring);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  // the last rows first: with a causal limit they have the most keys
  const int qt = (int)gridDim.x / p.Hq - 1 - (int)blockIdx.x / p.Hq, h = (int)blockIdx.x % p.Hq, b = blockIdx.y;
  const int row0 = qt * kRows, g = h / p.n_rep;
  const int rows = min(kRows, p.Lq - row0);
  // the tiles that the window leaves to these rows: the sinks' and the window's
  const int first = row0 + p.mask.coff, last = first + rows - 1, ntile = (p.Lk + kTile - 1) / kTile;
  const int w_sink = min(ntile, (p.mask.sinks + kTile - 1) / kTile);
  const int w_lo = max(w_sink, max(0, first - p.mask.window + 1) / kTile);
  const int w_hi = min(ntile, (max(0, p.mask.causal ? last + 1 : last + p.mask.window) + kTile - 1) / kTile);
  const int nt = w_sink + max(0, w_hi - w_lo);
  auto tile_key = [&](int c) { return (c < w_sink ? c : w_lo + c - w_sink) * kTile; };

  if (tid == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(sm.full + s, 1);
      mbar_init(sm.empty + s, kConsumers / 32);
    }
    fence_mbarrier_init();
    tc::prefetch_tensormap(&tm_k);
    tc::prefetch_tensormap(&tm_v);
  }
  __syncthreads();
  grid_dependency_wait();
  allow_dependents();
  if (warp >= kConsumers / 32) {
    tc::regs_dec<104>();
    if (warp == kConsumers / 32 && lane == 0) {
      bool ok = true;
      int it = 0;
      for (; it < nt && ok; ++it) {
        const int st = it % STAGES, use = it / STAGES;
        if (use > 0 && !(ok = mbar_wait(sm.empty + st, (use - 1) & 1, p.err))) break;
        unsigned char *kd = ring + st * 2 * TILEB;
        mbar_arrive_expect_tx(sm.full + st, 2 * TILEB);
        for (int c = 0; c < C::KB; ++c) {
          tc::tma_load_4d(kd + c * simt::kBox, &tm_k, c * 32, tile_key(it), g, b, sm.full + st);
          tc::tma_load_4d(kd + TILEB + c * simt::kBox, &tm_v, c * 32, tile_key(it), g, b, sm.full + st);
        }
      }
      // no copy may be in flight when the CTA exits, even if the consumers gave up
      for (int i = max(0, it - STAGES); i < it; ++i) mbar_wait(sm.full + i % STAGES, (i / STAGES) & 1, p.err);
    }
    return;
  }
  tc::regs_inc<200>();
  const simt::Place at(tid);
  const int kvl = load_kv_len(p.mask.kv_len, b, p.Lk, p.err, qt == 0 && h == 0 && tid == 0);
  const float *qb = p.q + (int64_t)b * p.qs[0] + (int64_t)h * p.qs[1];
#pragma unroll
  for (int u = tid; u < kRows * (D / 4); u += kConsumers) {
    const int r = u / (D / 4), d = (u % (D / 4)) * 4;
    float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
    if (r < rows) x = *reinterpret_cast<const float4 *>(qb + (int64_t)(row0 + r) * p.qs[2] + d);
    *reinterpret_cast<float4 *>(&sm.q[r][d]) = x;
  }
  // a thread's mask word: row tid / 2, half tid % 2 of the tile
  const int mrow = row0 + (tid >> 1), segq =
      p.mask.seg_q && tid < 2 * kRows && mrow < p.Lq ? __ldg(p.mask.seg_q + (int64_t)b * p.Lq + mrow) : -1;
  named_sync(1, kConsumers);

  float m[kRPG / 2], l[kRPG / 2];
  uint64_t o[kRPG][D / 64][2];
#pragma unroll
  for (int a = 0; a < kRPG / 2; ++a) {
    m[a] = -INFINITY;
    l[a] = 0.f;
  }
#pragma unroll
  for (int a = 0; a < kRPG; ++a)
#pragma unroll
    for (int c = 0; c < D / 64; ++c) o[a][c][0] = o[a][c][1] = 0ull;
  bool ok = true;
  int parts = 0;  // partial tiles so far
  for (int t = 0; t < nt; ++t) {
    const int st = t % STAGES, k0 = tile_key(t);
    const bool full = k0 + kTile <= min(p.Lk, kvl) && !p.mask.bits && !p.mask.seg_q &&
                      (!p.mask.causal || k0 + kTile - 1 <= first) &&
                      (k0 + kTile <= p.mask.sinks ||
                       (k0 > last - p.mask.window && (p.mask.causal || k0 + kTile <= first + p.mask.window)));
    const int mb = parts & 1;
    if (!full) {
      // (the other buffer's readers are past this barrier's predecessor)
      if (tid < 2 * kRows)
        sm.mask[mb][tid >> 1][tid & 1] =
            mrow < p.Lq ? mask_word(p.mask, b, mrow, k0 + 32 * (tid & 1), p.Lk, p.Lq, kvl, segq) : 0u;
      named_sync(1, kConsumers);
      ++parts;
    }
    if (ok) ok = __all_sync(0xffffffffu, mbar_wait(sm.full + st, (t / STAGES) & 1, p.err));
    const unsigned char *kt = ring + st * 2 * TILEB;
    // (values behind kv_len may hold anything)
    simt::tile<D, kRPG, C::QP>(ok, t & 1, &sm.q[0][0], kt, kt + TILEB, sm.sh, o, m, l, at, low_mask(kvl - k0),
                               low_mask(kvl - k0 - 32), [&](int a, int col, float s) {
                                 const bool see =
                                     full || ((sm.mask[mb][at.own<kRPG>(a)][col >> 5] >> (col & 31)) & 1u);
                                 return see ? s * p.scale_log2 : -INFINITY;
                               });
    __syncwarp();
    if (lane == 0) mbar_arrive(sm.empty + st);
  }
  float x[kRPG / 2][D / 64][4];
  simt::finish<D, kRPG>(sm.sh, o, l, x, at);
#pragma unroll
  for (int a = 0; a < kRPG / 2; ++a) {
    const int i = row0 + at.own<kRPG>(a);
    if (i >= p.Lq) continue;
    const float inv = ok && l[a] > 0.f ? 1.f / l[a] : 0.f;
    float *orow = p.out + (int64_t)b * p.os[0] + (int64_t)h * p.os[1] + (int64_t)i * p.os[2];
#pragma unroll
    for (int c = 0; c < D / 64; ++c)
      *reinterpret_cast<float4 *>(orow + at.tx * 4 + 64 * c) =
          make_float4(x[a][c][0] * inv, x[a][c][1] * inv, x[a][c][2] * inv, x[a][c][3] * inv);
    if (p.lse && at.tx == 0)
      p.lse[((int64_t)b * p.Hq + h) * p.Lq + i] = inv > 0.f ? (m[a] + log2f(l[a])) * kLn2 : -INFINITY;
  }
}

template <int D>
mgqa_status launch_t(const mgqa_args &a, const WinParams &p, cudaStream_t s) {
  using C = WinCfg<D>;
  CUtensorMap mk, mv;
  if (!make_tma_map_4d(&mk, MGQA_FP32, a.k, a.B, a.Hkv, a.Lk, D, a.k_stride, 32, kTile, true) ||
      !make_tma_map_4d(&mv, MGQA_FP32, a.v, a.B, a.Hkv, a.Lk, D, a.v_stride, 32, kTile, true))
    return fail(MGQA_ERR_CUDA, "cuTensorMapEncodeTiled failed");
  auto kern = prefill_window_f32_kernel<D>;
  static std::atomic<uint64_t> attr{0};
  const mgqa_status st = ensure_smem_attr(kern, C::smem, attr, "fp32 windowed prefill");
  if (st != MGQA_OK) return st;
  const cudaError_t e = launch_pdl(kern, dim3((unsigned)((a.Lq + kRows - 1) / kRows * a.Hq), a.B), dim3(kThreads), C::smem, s, mk, mv, p);
  if (e != cudaSuccess) return fail(MGQA_ERR_CUDA, "windowed prefill launch: %s", cudaGetErrorString(e));
  return MGQA_OK;
}

}  // namespace

mgqa_status launch_prefill_window_f32(const mgqa_args &a, const WindowRule &win, cudaStream_t s) {
  WinParams p{};
  p.q = static_cast<const float *>(a.q);
  p.out = static_cast<float *>(a.out);
  for (int t = 0; t < 3; ++t) {
    p.qs[t] = a.q_stride[t];
    p.os[t] = a.o_stride[t];
  }
  p.mask = MaskView{a.mask_bits, a.mask_stride_b, a.mask_stride_q, a.kv_len, a.seg_q, a.seg_k,
                    a.causal != 0, a.Lk - a.Lq, win.window, win.sinks};
  p.scale_log2 = a.scale * kLog2e;
  p.lse = a.lse; p.err = a.dev_error;
  p.Hq = a.Hq; p.Lq = a.Lq; p.Lk = a.Lk; p.n_rep = a.Hq / a.Hkv;
  return a.D == 64 ? launch_t<64>(a, p, s) : launch_t<128>(a, p, s);
}

}  // namespace mgqa
