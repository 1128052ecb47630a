// The 16-bit cache attention for more than 32 query rows per KV head (trees of
// drafted tokens over grouped heads; short calls of up to 64 rows excepted): the
// formulas of cache_attn.cu on the 5th-generation tensor cores.
//
// With R rows per KV head a key costs 4 R D operations for its 4 D bytes: at
// R = 256 the products take about as long as the reads, and mma.sync reaches a
// fraction of the tensor rate, so here the scores and outputs live in tensor
// memory. A CTA holds NT blocks of up to 128 query rows (row = draft * group +
// head, so a tile of keys serves every head of the group) and walks its run of
// the flat tile list (cache_sched.cuh). Two forms, by a rule at launch_d:
//   NT = 1: tiles of 64 keys, two score buffers, two CTAs an SM;
//   NT = 2: tiles of 128 keys, one CTA an SM.
// Warps:
//   warps 0, 3  : K and V, as boxes by TMA or row by row (cache_producer.cuh)
//   warp 1      : tensor memory, the MMA loop (one elected lane issues)
//   warp 2      : the query rows of the next piece, as soon as the last S of
//                 the current one is done, and its description for the others
//   warps 4..   : one softmax warpgroup per 128 rows (thread = row)
// Per tile n and row block t: S_t = Q_t K_n^T; softmax (running maximum, lazy
// rescale of O_t past 2^8) hands P_t over in tensor memory; O_t += P_t V_n.
// With two row blocks S_t(n+1) follows O_t += P_t V_n at once and the blocks
// take turns on the tensor cores and the softmax warps, as the heads in the
// prefill kernel. With one row block S(n+1) runs under the softmax of tile n (S
// behind P V, the chain of softmax, P V and S took longer than the reads).
// Between two pieces the softmax warpgroups read O_t out while the next query
// rows, K and V are on their way. (The softmax warps loading the rows themselves,
// between the pieces, cost ~4000 cycles a piece.) Values of keys that do not
// count (the end of a request, a missing page) are cleared in shared memory by
// the MMA warp before the product, on the tiles that have any.
// 61 drafts, 4 requests of 82020 slots on average, 32 heads over 8 (NT = 2): 270 us,
// 73 % of the copy rate and 0.64 of the bf16 rate with both needed at once (72 to 76 %
// from 75078 to 131004 slots; 6 % longer in runs of seconds); a tile
// takes ~4000 cycles against 3000 of reads and 2048 of products, the chain of P V,
// S and softmax of the prefill kernel. 24 drafts, 16 requests of 4739 slots on
// average (NT = 1): 67 us, 70 %; the rest is the start and the join.
// Every wait is bounded and reports MGQA_ERR_TIMEOUT.
#include <algorithm>
#include <cmath>

#include "cache_producer.cuh"
#include "tc_ptx.cuh"

namespace mgqa {
namespace {

constexpr int BM = 128;
constexpr int QBOX = BM * 128;  // bytes of 128 query rows x 64 columns, 128-byte swizzled
constexpr int kPieceRing = 4;  // a piece's slot is taken again after the S of the third piece behind it
constexpr int kOkRing = 8;     // tiles whose key masks are kept: K's producer is at most STAGES + 1 ahead of a softmax

struct TcCacheParams {
  CacheAttnParams a;
  int32_t box_rows;
  int32_t q_drafts;  // drafts of a block of up to 128 rows (each with all heads of the group)
};

template <int D, int NT>
struct Lay {
  static constexpr int SHIFT = NT == 1 ? 6 : 7, BN = 1 << SHIFT;  // keys of a tile
  static constexpr int CTAS = NT == 1 ? 2 : 1;                    // of an SM
  // registers: what the first warpgroup gives away goes to the softmax ones
  // (80 + 176 = 2 x 128, 104 + 2 x 200 = 3 x 168 a scheduler at launch)
  static constexpr int kDec = NT == 1 ? 80 : 104, kInc = NT == 1 ? 176 : 200;
  static constexpr int STAGES = D == 128 ? 2 : 4;
  static constexpr int KB = D / 64;
  static constexpr int BOX = BN * 128;  // bytes of a tile's 64 columns
  static constexpr int q_off = 0;
  static constexpr int k_off = q_off + NT * KB * QBOX;
  static constexpr int v_off = k_off + STAGES * KB * BOX;
  static constexpr int misc_off = v_off + STAGES * KB * BOX;
  static constexpr int threads = 128 * (1 + NT);
  static constexpr int ROWS = BM * NT;
  static constexpr int SB = NT == 1 ? 2 : 1;  // score buffers of a row block
  static constexpr uint32_t tmem_used = NT * (SB * BN + D);
  static constexpr uint32_t tmem_cols = tmem_used <= 256 ? 256 : 512;
  struct Misc {
    Drafts<kMaxDrafts> drafts;
    LocateScratch<threads> scratch;
    Piece pieces[kPieceRing];      // rp.nt < 0: no more
    uint64_t pready[kPieceRing], qfree;
    uint4 ok[kOkRing];  // which keys of a tile count
    uint64_t kfull[STAGES], vfull[STAGES], kempty[STAGES], vempty[STAGES];
    uint64_t sfull[NT * SB], pfull[NT * SB], odone[NT], ofree[NT], qfull[NT], drain;
    uint32_t tmem;
    int maxdepth;
  };
  static constexpr int smem = misc_off + (int)sizeof(Misc) + 1024;
  static_assert(CTAS * (smem + 1024) <= 228 * 1024 && CTAS * tmem_cols <= 512, "an SM holds the CTAs");
};

MGQA_DEV uint32_t all_of(const uint4 &w) { return w.x & w.y & w.z & w.w; }
MGQA_DEV uint32_t word_of(const uint4 &w, int i) { return i == 0 ? w.x : i == 1 ? w.y : i == 2 ? w.z : w.w; }

// One tile of one softmax row (thread = row) in tensor memory: see the
// prefill kernel's softmax_tile; the scale is not negative here.
// `pv_done`: phase `pv_parity` of that barrier tells that O holds every tile
// before this one (null: S of this tile was issued behind them).
template <typename T, int D, int BN, bool PARTIAL>
MGQA_DEV void softmax_row(uint32_t t_s, uint32_t t_o, const uint32_t (&mw)[4], float sl2, float &m_used, float &l,
                          uint64_t *pv_done, uint32_t pv_parity, int32_t *err) {
  uint32_t sr[BN];
  float mr;
  if constexpr (!PARTIAL) {
    float red[BN / 32];
#pragma unroll
    for (int c = 0; c < BN / 32; ++c)
      tc::tmem_ld32_red<true>(t_s + c * 32, *reinterpret_cast<uint32_t(*)[32]>(&sr[c * 32]), red[c]);
    tc::tmem_wait_ld();
    mr = fmaxf(red[0], red[1]);
    if constexpr (BN == 128) mr = fmaxf(mr, fmaxf(red[2], red[3]));
  } else {
#pragma unroll
    for (int c = 0; c < BN / 32; ++c) tc::tmem_ld32(t_s + c * 32, *reinterpret_cast<uint32_t(*)[32]>(&sr[c * 32]));
    tc::tmem_wait_ld();
    float mx[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) mx[k] = -INFINITY;
#pragma unroll
    for (int j = 0; j < BN; ++j)
      mx[j & 7] = fmaxf(mx[j & 7], (mw[j >> 5] >> (j & 31)) & 1u ? __uint_as_float(sr[j]) : -INFINITY);
#pragma unroll
    for (int k = 4; k > 0; k >>= 1)
#pragma unroll
      for (int u = 0; u < k; ++u) mx[u] = fmaxf(mx[u], mx[u + k]);
    mr = mx[0];
  }
  const float m_tile = mr == -INFINITY ? -INFINITY : mr * sl2;  // (a scale of 0 keeps "none")
  const float m_new = fmaxf(m_used, m_tile);
  bool rescale = false;
  float factor = 1.f;
  if (m_used == -INFINITY) {
    m_used = m_new;
  } else if (m_new - m_used > 8.f) {
    rescale = true;
    factor = tc::ex2(m_used - m_new);
    m_used = m_new;
    l *= factor;
  }
  if (__any_sync(0xffffffffu, rescale)) {
    if (pv_done) {
      mbar_wait(pv_done, pv_parity, err);
      __syncwarp();
      tc::fence_after_sync();
    }
#pragma unroll 1
    for (int c = 0; c < D / 32; ++c) {
      uint32_t o[32];
      tc::tmem_ld32(t_o + c * 32, o);
      tc::tmem_wait_ld();
#pragma unroll
      for (int j = 0; j < 32; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * factor);
      tc::tmem_st32(t_o + c * 32, o);
    }
    tc::tmem_wait_st();
  }
  const float mb = m_used == -INFINITY ? 0.f : m_used;
  const uint64_t sl2x2 = tc::pk2(sl2, sl2), nmb2 = tc::pk2(-mb, -mb);
  uint64_t acc[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) acc[k] = tc::pk2(0.f, 0.f);
#pragma unroll
  for (int c = 0; c < BN / 32; ++c) {
    uint32_t pk[16];
#pragma unroll
    for (int j = 0; j < 16; ++j) {
      const int col = c * 32 + 2 * j;
      const uint64_t y = tc::fma2(tc::pk2(__uint_as_float(sr[col]), __uint_as_float(sr[col + 1])), sl2x2, nmb2);
      float y0, y1;
      tc::upk2(y, y0, y1);
      float p0 = tc::ex2(y0), p1 = tc::ex2(y1);
      if (PARTIAL) {
        if (!((mw[c] >> (2 * j)) & 1u)) p0 = 0.f;
        if (!((mw[c] >> (2 * j + 1)) & 1u)) p1 = 0.f;
      }
      acc[j & 3] = tc::add2(acc[j & 3], tc::pk2(p0, p1));
      pk[j] = pack2<T>(p0, p1);
    }
    tc::tmem_st16(t_s + c * 16, pk);
  }
  acc[0] = tc::add2(acc[0], acc[1]);
  acc[2] = tc::add2(acc[2], acc[3]);
  acc[0] = tc::add2(acc[0], acc[2]);
  float s0, s1;
  tc::upk2(acc[0], s0, s1);
  l += s0 + s1;
  tc::tmem_wait_st();
}

// BOXES: K and V come as TMA boxes (else row by row: an instance of its own, the
// code of both in one cost 2 %).
template <typename T, int D, int NT, bool BOXES>
__global__ void __launch_bounds__(128 * (1 + NT), NT == 1 ? 2 : 1)
cache_attn_tc_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                     const __grid_constant__ CUtensorMap tm_kn, const __grid_constant__ CUtensorMap tm_vn,
                     const __grid_constant__ TcCacheParams tp) {
  using L = Lay<D, NT>;
  constexpr int KB = L::KB, STAGES = L::STAGES, ROWS = L::ROWS, BN = L::BN, BOX = L::BOX, kShift = L::SHIFT;
  const CacheAttnParams &p = tp.a;
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  unsigned char *smem = reinterpret_cast<unsigned char *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
  auto &sm = *reinterpret_cast<typename L::Misc *>(smem + L::misc_off);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;

  if (tid == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(sm.kfull + s, 1);
      mbar_init(sm.vfull + s, 1);
      mbar_init(sm.kempty + s, 1);
      mbar_init(sm.vempty + s, 1);
    }
    for (int t = 0; t < NT * L::SB; ++t) {
      mbar_init(sm.sfull + t, 1);
      mbar_init(sm.pfull + t, 128);
    }
    for (int t = 0; t < NT; ++t) {
      mbar_init(sm.odone + t, 1);
      mbar_init(sm.ofree + t, 128);
      mbar_init(sm.qfull + t, 1);
    }
    for (int i = 0; i < kPieceRing; ++i) mbar_init(sm.pready + i, 1);
    mbar_init(&sm.qfree, 1);
    mbar_init(&sm.drain, 1);
    fence_mbarrier_init();
    tc::prefetch_tensormap(&tm_q);
    if (BOXES) {
      tc::prefetch_tensormap(&tm_k);
      tc::prefetch_tensormap(&tm_v);
      tc::prefetch_tensormap(&tm_kn);
      tc::prefetch_tensormap(&tm_vn);
    }
  }
  if (warp == 1) tc::tmem_alloc(&sm.tmem, L::tmem_cols);
  if (warp == 2) touch_params(tp, lane);
  grid_dependency_wait();
  allow_dependents();  // lengths and tables are final from here on
  Walker walk;
  walk.start(p, locate<L::threads>(p, sm.scratch, gridDim.x, blockIdx.x, blockIdx.x == 0), blockIdx.x);
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tmem = sm.tmem;
  bool ok = true;
  Piece pc;
  int q_pieces = 0;
  auto role_end = [&]() {
    tc::fence_before_sync();
    named_sync(1, L::threads);
  };

  if (warp == 0 || warp == 3) {
    tc::regs_dec<L::kDec>();
    // ---------------- producers: K (warp 0) and V (warp 3) ----------------
    // (a box is issued by one lane at a time, ~80 cycles each: with pages of 8
    // slots the boxes of a whole tile took one warp longer than the reads)
    const bool of_v = warp == 3;
    const int br = tp.box_rows;
    uint64_t *full = of_v ? sm.vfull : sm.kfull, *empty = of_v ? sm.vempty : sm.kempty;
    unsigned char *buf = smem + (of_v ? L::v_off : L::k_off);
    const CUtensorMap *tm = of_v ? &tm_v : &tm_k, *tm_new = of_v ? &tm_vn : &tm_kn;
    int it = 0;  // tiles issued
    if constexpr (!BOXES) {
      // (the tensor cores read what the copies wrote only behind a proxy fence of the
      // copying threads, so a tile is told by its warp, when the next one has been
      // started, or ahead of a wait)
      RowFeed<KB, 2, kShift> feed;
      int told = 0;
      auto tell = [&](int upto) {
        fence_proxy_async_smem();
        __syncwarp();
        for (; told < upto; ++told)
          if (lane == 0) mbar_arrive(full + told % STAGES);
      };
      while (ok && walk.next(p, pc)) {
        feed.look_up(p, pc.rp, pc.b, pc.t0);
        for (int t = pc.t0; t < pc.t1; ++t) {
          const int st = it % STAGES, use = it / STAGES;
          if (use > 0) {
            const uint32_t parity = (uint32_t)(use - 1) & 1u;
            if (!__all_sync(0xffffffffu, mbar_test_wait(empty + st, parity))) {
              cp_async_wait<0>();
              tell(it);
              ok = __all_sync(0xffffffffu, mbar_wait(empty + st, parity, p.err));
              if (!ok) break;
            }
          }
          const auto now = feed;
          if (t + 1 < pc.t1) feed.look_up(p, pc.rp, pc.b, t + 1);
          uint32_t words[BN / 32];
          now.issue(p, pc.rp, pc.g, t, of_v, buf + st * KB * BOX, words);
          if (!of_v && lane == 0)
            sm.ok[it % kOkRing] = make_uint4(words[0], words[1], BN == 64 ? 0xffffffffu : words[BN / 32 - 2],
                                             BN == 64 ? 0xffffffffu : words[BN / 32 - 1]);
          cp_async_commit();
          cp_async_wait<1>();
          tell(it++);
        }
      }
      cp_async_wait<0>();  // (also: no copy is in flight when the CTA exits)
      tell(it);
    } else {
      BoxPages pages;
      while (ok && walk.next(p, pc)) {
        const RowPlan &rp = pc.rp;
        pages.start(p, pc, kShift, br);
        for (int t = pc.t0; t < pc.t1; ++t, ++it) {
          const int page = pages.page(p, pc, kShift, br, t);  // (lane i: box i of the tile)
          int kind;
          const int k0 = first_key(rp, t, kShift, kind);
          const int j0 = k0 + lane * br;
          uint32_t mine[4] = {0u, 0u, 0u, 0u};  // (a tile of 64 keys has two words)
          bool take = false;
          if (kind) {
            take = lane == 0 && rp.live > k0;
            if (lane == 0)
#pragma unroll
              for (int w = 0; w < BN / 32; ++w) mine[w] = low_mask(rp.live - k0 - 32 * w);
          } else if (page >= 0) {
            take = true;
#pragma unroll
            for (int w = 0; w < BN / 32; ++w) {
              const int j = k0 + 32 * w;
              mine[w] = low_mask(rp.n - j) & (~low_mask(rp.lo - j) | low_mask(rp.s_end - j)) & low_mask(j0 + br - j) &
                        ~low_mask(j0 - j);
            }
          } else if (page == -1) {
            report_error(p.err, MGQA_ERR_INVALID_ARG);
          }
          uint4 words;
          if (!of_v) {
            words.x = __reduce_or_sync(0xffffffffu, mine[0]);
            words.y = __reduce_or_sync(0xffffffffu, mine[1]);
            words.z = BN == 64 ? 0xffffffffu : __reduce_or_sync(0xffffffffu, mine[2]);
            words.w = BN == 64 ? 0xffffffffu : __reduce_or_sync(0xffffffffu, mine[3]);
          }
          const uint32_t bytes = (uint32_t)(__popc(__ballot_sync(0xffffffffu, take)) * (kind ? BN : br) * 128 * KB);
          const int st = it % STAGES, use = it / STAGES;
          const int slot = kind ? k0 : slot_in_page(p, j0), z = kind ? pc.b : page;
          unsigned char *dst = buf + st * KB * BOX + (kind ? 0 : lane * br * 128);
          if (use > 0) ok = __all_sync(0xffffffffu, mbar_wait(empty + st, (use - 1) & 1, p.err));
          if (!ok) break;
          if (lane == 0) {
            if (!of_v) sm.ok[it % kOkRing] = words;
            mbar_arrive_expect_tx(full + st, bytes);
          }
          __syncwarp();
          if (take)
#pragma unroll
            for (int c = 0; c < KB; ++c)
              tc::tma_load_4d(dst + c * BOX, kind ? tm_new : tm, c * 64, slot, pc.g, z, full + st);
        }
      }
      // no copy may be in flight when the CTA exits (only this warp arms these full
      // barriers: the last armed phase of each is the newest it can reach)
      __syncwarp();
      for (int i = max(0, it - STAGES); i < it; ++i) mbar_wait(full + i % STAGES, (i / STAGES) & 1, p.err);
      __syncwarp();
    }
    role_end();
  } else if (warp == 1) {
    tc::regs_dec<L::kDec>();
    // ---------------- MMA issuer ----------------
    const bool leader = tc::elect_one();
    constexpr bool kBf16 = !__is_same(T, __half);
    constexpr uint32_t id_s = tc::idesc_16bit(BM, BN, 0, 0, kBf16);
    constexpr uint32_t id_pv = tc::idesc_16bit(BM, D, 0, 1, kBf16);
    const uint32_t sb = smem_u32(smem);
    const uint64_t qd0 = tc::sw128_desc(sb + L::q_off, 16, 1024);
    const uint64_t kd0 = tc::sw128_desc(sb + L::k_off, 16, 1024);
    const uint64_t vd0 = tc::sw128_desc(sb + L::v_off, BOX, 1024);
    constexpr uint64_t kTileStep = (uint64_t)(KB * BOX) >> 4, kQStep = (uint64_t)(KB * QBOX) >> 4;
    auto wait = [&](uint64_t *bar, uint32_t parity) {
      ok = __all_sync(0xffffffffu, ok && mbar_wait(bar, parity, p.err));
      return ok;
    };
    // S of row block t, into score buffer sb
    auto issue_s = [&](int t, int sb, int st, int k0, int k1, bool last) {
      const uint64_t qd = qd0 + (uint64_t)t * kQStep, kd = kd0 + (uint64_t)st * kTileStep;
      if (leader) {
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          if (kk < k0 || kk >= k1) continue;
          const uint64_t qo = (uint64_t)((kk / 4) * QBOX + (kk % 4) * 32) >> 4;
          const uint64_t ko = (uint64_t)((kk / 4) * BOX + (kk % 4) * 32) >> 4;
          tc::mma_ss(tmem + (t + sb) * BN, qd + qo, kd + ko, id_s, kk > 0 ? 1u : 0u);
        }
        if (k1 == D / 16) {
          tc::mma_commit(sm.sfull + t + sb);
          if (t == NT - 1) tc::mma_commit(sm.kempty + st);
          if (t == NT - 1 && last) tc::mma_commit(&sm.qfree);  // the piece's query rows are read
        }
      }
      __syncwarp();
    };
    auto issue_pv = [&](int t, int sb, int st, int k0, int k1, bool first) {
      const uint64_t vd = vd0 + (uint64_t)st * kTileStep;
      if (leader) {
#pragma unroll
        for (int kk = 0; kk < BN / 16; ++kk) {
          if (kk < k0 || kk >= k1) continue;
          tc::mma_ts(tmem + NT * L::SB * BN + t * D, tmem + (t + sb) * BN + kk * 8, vd + (uint64_t)(kk * 2048 >> 4), id_pv,
                     (!first || kk > 0) ? 1u : 0u);
        }
      }
      __syncwarp();
    };
    constexpr int kHalfPV = BN / 32, kLateS = D / 16 - 1;
    int it = 0;  // tiles of the pieces before this one
    for (int piece = 0; ok && walk.next(p, pc); ++piece) {
      const int nk = pc.t1 - pc.t0;
      if (!wait(sm.kfull + it % STAGES, (it / STAGES) & 1)) break;
      for (int t = 0; t < NT && ok; ++t) {
        if (!wait(sm.qfull + t, piece & 1)) break;
        tc::fence_after_sync();
        issue_s(t, it % L::SB, it % STAGES, 0, D / 16, nk == 1);
      }
      if (!ok || !wait(sm.vfull + it % STAGES, (it / STAGES) & 1)) break;
      bool p0_seen = false;
      for (int n = 0; n < nk && ok; ++n) {
        const int at = it + n, st1 = (at + 1) % STAGES;
        const uint32_t par1 = (uint32_t)((at + 1) / STAGES) & 1u;
        const int sv = at % STAGES;
        const bool has_next = n + 1 < nk;
        {  // values of keys that do not count: cleared (their rows may hold anything,
           // but for those behind the drafts, which a box fills with zeros)
          const uint4 okw = sm.ok[at % kOkRing];
          if (all_of(okw) != 0xffffffffu) {
            int kind;
            const int k0 = first_key(pc.rp, pc.t0 + n, kShift, kind);
            const int rows = BOXES && kind && pc.rp.live > k0 ? p.T - k0 : BN;
#pragma unroll
            for (int w = 0; w < BN / 32; ++w) {
              const uint32_t clear = ~word_of(okw, w) & low_mask(rows - 32 * w);
              if (clear)  // 16-byte pieces (the swizzle permutes them within a row)
#pragma unroll
                for (int u = 0; u < D / 8; ++u) {
                  const int r = (u * 32 + lane) / (D / 8), c = (u * 32 + lane) % (D / 8);
                  if ((clear >> r) & 1u)
                    *reinterpret_cast<uint4 *>(smem + L::v_off + (sv * KB + (c >> 3)) * BOX + (32 * w + r) * 128 +
                                               (c & 7) * 16) = make_uint4(0u, 0u, 0u, 0u);
                }
            }
            fence_proxy_async_smem();
            __syncwarp();
          }
        }
        if constexpr (NT == 1) {
          // the next S goes out ahead of this tile's softmax result
          if (has_next) {
            if (!wait(sm.kfull + st1, par1)) break;
            tc::fence_after_sync();
            issue_s(0, (at + 1) & 1, st1, 0, D / 16, n + 2 == nk);
          }
          // (a barrier per score buffer: P(n+1), which no longer waits for P V of tile n,
          // would otherwise be able to complete a second phase ahead of this wait)
          if (!wait(sm.pfull + (at & 1), (at >> 1) & 1)) break;
          if (n == 0 && piece > 0 && !wait(sm.ofree, (piece - 1) & 1)) break;
          tc::fence_after_sync();
          issue_pv(0, at & 1, sv, 0, BN / 16, n == 0);
          if (leader) {
            tc::mma_commit(sm.vempty + sv);
            if (!has_next) tc::mma_commit(sm.odone);
          }
          __syncwarp();
          if (has_next && !wait(sm.vfull + st1, par1)) break;
        } else {
          bool p1_seen = false;
          for (int t = 0; t < NT && ok; ++t) {
            if (!(t == 0 ? p0_seen : p1_seen) && !wait(sm.pfull + t, at & 1)) break;
            if (n == 0 && piece > 0 && !wait(sm.ofree + t, (piece - 1) & 1)) break;
            tc::fence_after_sync();
            issue_pv(t, 0, sv, 0, kHalfPV, n == 0);
            if (has_next) {  // K of the next tile before its first S, V before the next P.V
              if (t == 0 && !wait(sm.kfull + st1, par1)) break;
              if (t == NT - 1 && !wait(sm.vfull + st1, par1)) break;
              tc::fence_after_sync();
            }
            issue_pv(t, 0, sv, kHalfPV, BN / 16, n == 0);
            if (leader) {
              if (!has_next) tc::mma_commit(sm.odone + t);
              if (t == NT - 1) tc::mma_commit(sm.vempty + sv);
            }
            __syncwarp();
            if (has_next) {
              issue_s(t, 0, st1, 0, kLateS, false);
              if (t == NT - 1) p0_seen = __all_sync(0xffffffffu, mbar_test_wait(sm.pfull, (at + 1) & 1));
              else p1_seen = __all_sync(0xffffffffu, mbar_test_wait(sm.pfull + 1, at & 1));
              issue_s(t, 0, st1, kLateS, D / 16, n + 2 == nk);
            }
          }
        }
      }
      it += nk;
    }
    // the last release of every stage has landed before the CTA exits; after a
    // wait that gave up, every MMA issued completes before tensor memory is freed
    for (int i = max(0, it - STAGES); i < it && ok; ++i)
      wait(sm.kempty + i % STAGES, (i / STAGES) & 1) && wait(sm.vempty + i % STAGES, (i / STAGES) & 1);
    if (!ok) {
      if (leader) tc::mma_commit(&sm.drain);
      __syncwarp();
      mbar_wait(&sm.drain, 0, p.err);
    }
    __syncwarp();
    role_end();
    tc::fence_after_sync();
    tc::tmem_dealloc(tmem, L::tmem_cols);
  } else if (warp == 2) {
    tc::regs_dec<L::kDec>();
    // ---------------- query rows and piece descriptions ----------------
    bool more = true;
    if (lane == 0) tell_cut(p, blockIdx.x, nullptr);
    for (int piece = 0; more; ++piece) {
      more = walk.next(p, pc);
      if (more && lane == 0) tell_cut(p, blockIdx.x, &pc);
      // (the slot is free: its piece's query rows were overwritten long ago)
      if (ok && piece > 0) ok = __all_sync(0xffffffffu, mbar_wait(&sm.qfree, (piece - 1) & 1, p.err));
      if (!ok) more = false;
      if (lane == 0) {
        if (!more) pc.rp.nt = -1;
        sm.pieces[piece % kPieceRing] = pc;
        mbar_arrive(sm.pready + piece % kPieceRing);
        if (more) {
          // block t: its drafts, each with the group's heads as consecutive rows
          const int drafts = tp.q_drafts, first = pc.rb * drafts * NT;
#pragma unroll
          for (int t = 0; t < NT; ++t) {
            mbar_arrive_expect_tx(sm.qfull + t, (uint32_t)(KB * drafts * p.n_rep * 128));
#pragma unroll
            for (int c = 0; c < KB; ++c)
              tc::tma_load_5d(smem + L::q_off + (t * KB + c) * QBOX, &tm_q, c * 64, 0, first + t * drafts, pc.g, pc.b,
                              sm.qfull + t);
          }
          q_pieces = piece + 1;
        }
      }
      __syncwarp();
    }
    // no copy may be in flight when the CTA exits
    if (q_pieces > 0)
      for (int t = 0; t < NT; ++t) mbar_wait(sm.qfull + t, (q_pieces - 1) & 1, p.err);
    __syncwarp();
    role_end();
  } else {
    tc::regs_inc<L::kInc>();
    // ---------------- softmax warpgroup t ----------------
    const int t = (warp - 4) >> 2, quarter = warp & 3;
    const int r = quarter * 32 + lane;  // row of the tile
    const int stid = tid - 128;         // thread among the softmax warps
    const uint32_t lanes = (uint32_t)(quarter * 32) << 16;
    const uint32_t t_s0 = tmem + lanes + t * BN, t_o = tmem + lanes + NT * L::SB * BN + t * D;
    const float sl2 = p.scale_log2;
    int it = 0, staged = -1;
    for (int piece = 0;; ++piece) {
      if (ok) ok = mbar_wait(sm.pready + piece % kPieceRing, (piece / kPieceRing) & 1, p.err);
      ok = __all_sync(0xffffffffu, ok);
      const Piece &pc = sm.pieces[piece % kPieceRing];
      if (!ok || pc.rp.nt < 0) break;
      const RowPlan &rp = pc.rp;
      const PieceOut po = out_of(p, pc, blockIdx.x);
      const int brow = t * tp.q_drafts * p.n_rep + r;  // row of the blocks
      const int row = po.row0 + brow;
      const bool has_row = r < tp.q_drafts * p.n_rep && brow < po.rows;
      const bool need_drafts = p.tree && (p.window != kNoWindow || pc.t1 > rp.np);
      if (need_drafts && staged != pc.b) {
        named_sync(2, 128 * NT);  // the masks of an earlier request are no longer read
        if (stid == 0) sm.maxdepth = 0;
        stage_drafts(p, sm.drafts, pc.b, rp.live, stid, 128 * NT);
        named_sync(2, 128 * NT);
        int md = 0;
        for (int x = stid; x < rp.live; x += 128 * NT) md = max(md, sm.drafts.depth[x]);
        if (md) atomicMax(&sm.maxdepth, md);
        named_sync(2, 128 * NT);
        staged = pc.b;
      }
      RowSight rs;
      rs.t = row / p.n_rep;
      rs.ok = has_row && (!p.tree || rs.t < rp.live);
      const int pt = p.tree ? rp.n + (need_drafts && rs.ok ? sm.drafts.depth[rs.t] : 0) : rp.n - 1;
      rs.lo = pt - p.window + 1;
      const int lo_all = rp.n + (p.tree ? (need_drafts ? sm.maxdepth : 0) : -1) - p.window + 1;
      float m_used = -INFINITY, l = 0.f;
      const int t1 = pc.t1;
      for (int i = pc.t0; i < t1; ++i, ++it) {
        // (a barrier per score buffer: S(n+1) may complete before S(n) is waited for)
        const int sb = it % L::SB;
        const uint32_t t_s = t_s0 + sb * BN;
        if (ok) ok = mbar_wait(sm.sfull + t + sb, (it / L::SB) & 1, p.err);
        ok = __all_sync(0xffffffffu, ok);
        if (ok) {  // after a failed wait, tensor memory is left alone
          int kind;
          const int k0 = first_key(rp, i, kShift, kind);
          const uint4 okw = sm.ok[it % kOkRing];
          const bool full = !kind && all_of(okw) == 0xffffffffu && (k0 >= lo_all || k0 + BN <= min(p.sinks, rp.s_end));
          tc::fence_after_sync();
          // (a rescale follows an earlier tile of the piece; its P V releases that tile's V stage)
          uint64_t *pv_done = L::SB > 1 ? sm.vempty + (it - 1 + STAGES) % STAGES : nullptr;
          const uint32_t pv_parity = (uint32_t)((it - 1) / STAGES) & 1u;
          uint32_t mw[4] = {0u, 0u, 0u, 0u};
          if (full) {
            softmax_row<T, D, BN, false>(t_s, t_o, mw, sl2, m_used, l, pv_done, pv_parity, p.err);
          } else {
#pragma unroll
            for (int w = 0; w < BN / 32; ++w) {
              const int j = k0 + 32 * w;
              uint32_t x = rs.ok ? word_of(okw, w) : 0u;
              if (!kind) {
                x &= ~low_mask(rs.lo - j) | low_mask(p.sinks - j);
              } else if (x) {
                x &= sm.drafts.see[rs.t][j >> 5];
                if (p.window != kNoWindow)
                  for (uint32_t y = x; y; y &= y - 1) {
                    const int s = __ffs(y) - 1, ps = rp.n + sm.drafts.depth[j + s];
                    if (ps < rs.lo && ps >= p.sinks) x &= ~(1u << s);
                  }
              }
              mw[w] = x;
            }
            softmax_row<T, D, BN, true>(t_s, t_o, mw, sl2, m_used, l, pv_done, pv_parity, p.err);
          }
          tc::fence_before_sync();
        }
        mbar_arrive(sm.pfull + t + sb);
      }
      // ---- the piece's rows: O out of tensor memory, finished or as a partial result
      if (ok) ok = mbar_wait(sm.odone + t, piece & 1, p.err);
      ok = __all_sync(0xffffffffu, ok);
      tc::fence_after_sync();
      const bool none = !ok || !rs.ok || m_used == -INFINITY;
      const float m = none ? -INFINITY : m_used, lr = none ? 0.f : l;
      const RowOut<T, D, ROWS> dst(p, po, has_row ? brow : 0, m, lr, has_row);
#pragma unroll
      for (int c = 0; c < D / 32; ++c) {
        uint32_t x[32];
        if (ok) {
          tc::tmem_ld32(t_o + c * 32, x);
          tc::tmem_wait_ld();
        }
        if (has_row)
#pragma unroll
          for (int j = 0; j < 32; j += 8) {
            float o[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) o[e] = none ? 0.f : __uint_as_float(x[j + e]);
            dst.put(c * 32 + j, o);
          }
      }
      tc::fence_before_sync();
      mbar_arrive(sm.ofree + t);
    }
    role_end();
  }
}

template <typename T, int D, int NT, bool BOXES>
mgqa_status launch_b(TcCacheParams tp, mgqa_dtype dt, const CUtensorMap (&maps)[4], const CacheAttnLaunch &how,
                     cudaStream_t s) {
  using L = Lay<D, NT>;
  auto kern = cache_attn_tc_kernel<T, D, NT, BOXES>;
  static std::atomic<uint64_t> attr{0};
  const mgqa_status st = ensure_smem_attr(kern, L::smem, attr, "cache attention kernel");
  if (st != MGQA_OK) return st;
  CacheAttnParams &p = tp.a;
  tp.q_drafts = BM / p.n_rep;
  p.block_rows = NT * tp.q_drafts * p.n_rep;
  p.RB = (p.R + p.block_rows - 1) / p.block_rows;
  p.tile_shift = L::SHIFT;
  // q [B][Hkv][T][group][D]: a box is a block's drafts with the heads of one group
  CUtensorMap mq;
  const int64_t dims[5] = {D, p.n_rep, p.T, p.Hkv, p.B};
  const int64_t strides[4] = {p.qs[1], p.qs[2], p.qs[1] * p.n_rep, p.qs[0]};
  const int box[5] = {64, p.n_rep, tp.q_drafts, 1, 1};
  if (!make_tma_map(&mq, dt, p.q, 5, dims, strides, box, true))
    return fail(MGQA_ERR_CUDA, "cuTensorMapEncodeTiled failed for q");
  p.lead = NT == 1 ? 4 : 8;  // (3 and 6 are within 2 % on NT = 1; 3 costs 9 % with two blocks and one request)
  p.min_run = 4;
  const int64_t tiles = (int64_t)p.B * p.Hkv * p.RB * (most_tiles(p) + p.lead);
  const int grid = (int)std::max<int64_t>(1, std::min<int64_t>(std::min(how.sms, kCacheAttnMaxCtas / 2) * L::CTAS, tiles));
  set_partials(p, how.workspace, grid, L::ROWS, D);
  const cudaError_t e = launch_pdl(kern, dim3(grid), dim3(L::threads), L::smem, s, mq, maps[0], maps[1], maps[2],
                                   maps[3], tp);
  if (e != cudaSuccess) return fail(MGQA_ERR_CUDA, "cache attention launch: %s", cudaGetErrorString(e));
  return launch_cache_merge(p, dt, D, L::ROWS, grid, s);
}

template <typename T, int D, int NT>
mgqa_status launch_t(TcCacheParams tp, mgqa_dtype dt, const CacheAttnLaunch &how, cudaStream_t s) {
  CUtensorMap maps[4];
  if (!cache_attn_maps(tp.a, dt, D, Lay<D, NT>::BN, maps, tp.box_rows))
    return fail(MGQA_ERR_CUDA, "cuTensorMapEncodeTiled failed for the cache");
  return tp.box_rows ? launch_b<T, D, NT, true>(tp, dt, maps, how, s) : launch_b<T, D, NT, false>(tp, dt, maps, how, s);
}

template <typename T, int D>
mgqa_status launch_d(const TcCacheParams &tp, mgqa_dtype dt, const CacheAttnLaunch &how, cudaStream_t s) {
  // More than 128 rows: two blocks a CTA share every key tile, one CTA an SM; or
  // one block a CTA, two CTAs an SM, each reading the keys (mostly from the L2)
  // but covering for one another between units. The second is ahead while the
  // call is not long (64 drafts, 32 heads over 8: one request of up to 4096 tokens
  // 22.0 and 14.9 us; 16 of up to 2048 57 and 48; 16 of up to 8192 99 and 108; 4 of
  // up to 131072 266 and 396; D = 64, 16 of about 8100 117 and 113). The lengths are
  // on the device, so the capacity decides: one request of 4000 tokens takes 18.4 us
  // in a table for 4096 slots and 24.3 in one for 131072.
  CacheAttnParams q = tp.a;
  q.tile_shift = 6;
  const int64_t reads = (int64_t)q.B * q.Hkv * most_tiles(q) * (kTile * D * 4);
  const bool one = q.T <= BM / q.n_rep || reads <= ((int64_t)(D == 64 ? 384 : 192) << 20);
  return one ? launch_t<T, D, 1>(tp, dt, how, s) : launch_t<T, D, 2>(tp, dt, how, s);
}

}  // namespace

bool cache_attn_tc_takes(const CacheAttnParams &p) {
  return p.n_rep <= BM && p.scale_log2 >= 0.f && plain_strides(p.qs, p.B, p.Hq, p.T);
}

mgqa_status launch_cache_attn_tc(const CacheAttnParams &p, mgqa_dtype dt, int D, const CacheAttnLaunch &how,
                                 cudaStream_t s) {
  TcCacheParams tp{};
  tp.a = p;
  if (dt == MGQA_BF16)
    return D == 64 ? launch_d<__nv_bfloat16, 64>(tp, dt, how, s) : launch_d<__nv_bfloat16, 128>(tp, dt, how, s);
  return D == 64 ? launch_d<__half, 64>(tp, dt, how, s) : launch_d<__half, 128>(tp, dt, how, s);
}

}  // namespace mgqa
