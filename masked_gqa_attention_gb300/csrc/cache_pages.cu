// The cache's own steps: appending rows, forking / freeing / reserving requests
// of pages, and packing the pool. All of them move rows as they are; the
// floor is one read and one write of every row moved.
//
// append: one pass, a block per (layer, request, run of rows); a thread has
//   one 16-byte piece of K and of V in flight, read in the order in which a
//   projection leaves them ([T][Hkv][D]) and written as whole D-rows. (32768 rows
//   of 8 x 128 bf16: eight pieces a thread 64.6 us, four 51.7, two 45.5, one 43:
//   smaller blocks overlap their look-ups with other blocks' copies.)
// fork and compact: the page bookkeeping is integer work on a few arrays whose
//   result every block needs, so it runs ahead of the copies in kernels of its
//   own, joined by programmatic dependent launches:
//     fork    -- gather (stages the sources' table rows, gives back and takes
//                shares by integer atomics, whose order cannot matter; a block
//                per pair), plan (one block: free pages as a bitmap in shared
//                memory, requests and free pages matched by prefix sums), apply
//                (table rows, lengths, and the copies). (The planning block
//                gathering by itself, a launch less: no call was faster. 4 pairs
//                of 33 entries 9.5 us against 8.8, of 252 14.5 against 8.9;
//                32 pairs of 64 12.9 against 11.2.)
//     compact -- plan (one block: the used pages as a bitmap, moves by prefix
//                sums over its words) and apply (copies, table, counts).
//   One block is enough for the plan: a pool of 2^16 pages is 256 KB of counts.
#include <algorithm>

#include "common.cuh"
#include "internal.h"

namespace mgqa {
namespace {

// K and V of a cache as bytes.
struct Pool {
  char *k, *v;
  int64_t ks[4], vs[4];  // layer, page, head, slot strides in bytes
  int32_t layers, num_pages, Hkv, page_size, pieces;  // pieces: 16-byte pieces of a D-row
  int32_t rows, max_pages;
  int32_t *table;
  int64_t table_stride;
  int32_t *kv_len, *ref, *err;
};

Pool pool_of(const mgqa_cache &c) {
  const int64_t es = c.dtype == MGQA_FP32 ? 4 : 2;
  Pool p{};
  p.k = static_cast<char *>(c.k);
  p.v = static_cast<char *>(c.v);
  for (int t = 0; t < 4; ++t) {
    p.ks[t] = c.k_stride[t] * es;
    p.vs[t] = c.v_stride[t] * es;
  }
  p.layers = c.layers; p.num_pages = c.num_pages; p.Hkv = c.Hkv; p.page_size = c.page_size;
  p.pieces = (int32_t)(c.D * es / 16);
  p.rows = c.rows; p.max_pages = c.max_pages;
  p.table = c.page_table; p.table_stride = c.table_stride;
  p.kv_len = c.kv_len; p.ref = c.ref; p.err = c.dev_error;
  return p;
}

MGQA_DEV int valid_page(const Pool &p, int e) { return (unsigned)e < (unsigned)p.num_pages ? e : -1; }

// ---- append -------------------------------------------------------------------

constexpr int kAppendThreads = 256;

struct AppendParams {
  Pool c;
  const char *kn, *vn;
  int64_t kns[4], vns[4];  // layer, batch, head, row strides in bytes
  int32_t T;
  int32_t block_rows;  // new rows of a block
  const int32_t *index, *count;
  int32_t *kv_len_out;
  // kv_len_out shares no 128-byte line with kv_len, count, index or the page table.
  // Otherwise those are read past the L1: the next kernel is resident before this one
  // ends, and a line left there could give it an old kv_len_out. (kv_len alone read
  // so always: 32768 rows take 46 us, not 42.)
  int32_t ints_apart;
};

__global__ void __launch_bounds__(kAppendThreads)
append_kernel(const __grid_constant__ AppendParams p) {
  const Pool &c = p.c;
  const int b = blockIdx.y, layer = blockIdx.z;
  grid_dependency_wait();
  allow_dependents();
  const int64_t cap = c.table ? (int64_t)c.max_pages * c.page_size : c.page_size;
  const auto load = [&](const int32_t *x) { return p.ints_apart ? __ldg(x) : __ldcg(x); };
  const int n = load(c.kv_len + b);
  const int cnt = p.count ? load(p.count + b) : p.T;
  const bool bad = n < 0 || cnt < 0 || cnt > p.T || (int64_t)n + cnt > cap;
  // the block's rows from t0 on, all heads of each. Without a count the new rows
  // are read ahead of what tells where they go (the length, then the page).
  const int per = c.Hkv * c.pieces;
  const int t0 = (int)blockIdx.x * p.block_rows, rows = min(p.block_rows, p.T - t0);
  for (int i = threadIdx.x; i < rows * per; i += kAppendThreads) {
    const int tl = i / per, rem = i - tl * per, t = t0 + tl;
    const int h = rem / c.pieces, piece = rem - h * c.pieces;
    if (p.count && (bad || t >= cnt)) break;
    const int from = p.index ? load(p.index + (int64_t)b * p.T + t) : t;
    const bool has = (unsigned)from < (unsigned)p.T;
    uint4 kx, vx;
    if (has) {
      kx = __ldcs(reinterpret_cast<const uint4 *>(p.kn + layer * p.kns[0] + b * p.kns[1] + h * p.kns[2] +
                                                  (int64_t)from * p.kns[3] + piece * 16));
      vx = __ldcs(reinterpret_cast<const uint4 *>(p.vn + layer * p.vns[0] + b * p.vns[1] + h * p.vns[2] +
                                                  (int64_t)from * p.vns[3] + piece * 16));
    }
    if (bad) break;
    const int j = n + t;
    int page = b, slot = j;
    if (c.table) {
      const int pi = j / c.page_size;
      page = valid_page(c, load(c.table + (int64_t)b * c.table_stride + pi));
      slot = j - pi * c.page_size;
    }
    if (has && page >= 0) {
      __stcs(reinterpret_cast<uint4 *>(c.k + layer * c.ks[0] + (int64_t)page * c.ks[1] + h * c.ks[2] +
                                       (int64_t)slot * c.ks[3] + piece * 16), kx);
      __stcs(reinterpret_cast<uint4 *>(c.v + layer * c.vs[0] + (int64_t)page * c.vs[1] + h * c.vs[2] +
                                       (int64_t)slot * c.vs[3] + piece * 16), vx);
    } else if (layer == 0 && rem == 0) {
      report_error(c.err, MGQA_ERR_INVALID_ARG);
    }
  }
  if (blockIdx.x == 0 && layer == 0 && threadIdx.x == 0) {
    if (bad) report_error(c.err, MGQA_ERR_INVALID_ARG);
    p.kv_len_out[b] = bad ? n : n + cnt;
  }
}

// ---- append to a cache in 4 bits -----------------------------------------------------

// As append, the rows quantised on the way (cache_q4.cuh has the record). A thread
// has eight features of a row of K and of V; a group's extremes are found between
// its 4 (D = 64: 2) threads, in the rows' own type, least and (negated) greatest in
// one word. Every step is one fp32 operation, so the codes are the same wherever they
// are computed:
//   least = fp16(min), scale = fp16((max - least) fl(1/15)), both within +-65504 and
//   without a negative zero; u = clamp(rint((x - least) / scale), 0, 15), 0 where
//   scale is 0.
// Moving rows is all a cache needs, but a row's 16 quotients a thread are the time:
// they come from a reciprocal. 32768 rows of 8 x 128 bf16 take 56 us (150 with
// divisions; the reads and writes are 26): 410 instructions a warp of 32 x 16 values,
// 85 % of the issue slots.
struct Q4Params {
  AppendParams a;
  uint32_t kstep[4], vstep[4];    // cache: layer, page, head, slot in 16-byte pieces
  uint32_t knstep[4], vnstep[4];  // new rows: layer, batch, head, row
  int32_t alike;                  // k's and v's steps agree
  int32_t page_shift;             // of a power of two, else -1
  uint32_t by_heads;              // x / Hkv = x * by_heads >> 32 for x < 2^16 (and Hkv > 1)
};
struct Q4Piece {
  uint32_t codes;  // of the thread's eight features, in the record's order
  uint32_t par;    // scale and least value of its group
};

// Eight values as they lie in memory.
template <typename T>
struct Eight {
  uint4 w[sizeof(T) / 2];
  MGQA_DEV void load(const char *p) {
#pragma unroll
    for (int i = 0; i < (int)sizeof(T) / 2; ++i) w[i] = __ldcs(reinterpret_cast<const uint4 *>(p) + i);
  }
  MGQA_DEV void values(float (&x)[8]) const {
    if constexpr (sizeof(T) == 4) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        x[4 * i] = __uint_as_float(w[i].x); x[4 * i + 1] = __uint_as_float(w[i].y);
        x[4 * i + 2] = __uint_as_float(w[i].z); x[4 * i + 3] = __uint_as_float(w[i].w);
      }
    } else {
      unpack16_t<T>(w[0], x);
    }
  }
};

MGQA_DEV uint32_t min_pair(uint32_t a, uint32_t b, __nv_bfloat16) {
  const __nv_bfloat162 r = __hmin2(*reinterpret_cast<const __nv_bfloat162 *>(&a), *reinterpret_cast<const __nv_bfloat162 *>(&b));
  return *reinterpret_cast<const uint32_t *>(&r);
}
MGQA_DEV uint32_t min_pair(uint32_t a, uint32_t b, __half) {
  const __half2 r = __hmin2(*reinterpret_cast<const __half2 *>(&a), *reinterpret_cast<const __half2 *>(&b));
  return *reinterpret_cast<const uint32_t *>(&r);
}

// The least and the greatest value of a group. (Whole warps.)
template <typename T, int D>
MGQA_DEV void extremes(const Eight<T> &e, const float (&x)[8], float &lo, float &hi) {
  if constexpr (sizeof(T) == 4) {
    lo = hi = x[0];
#pragma unroll
    for (int i = 1; i < 8; ++i) {
      lo = fminf(lo, x[i]);
      hi = fmaxf(hi, x[i]);
    }
#pragma unroll
    for (int o = 1; o < D / 32; o <<= 1) {
      lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, o));
      hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, o));
    }
  } else {
    constexpr uint32_t kSigns = 0x80008000u;
    const uint4 &w = e.w[0];
    const uint32_t a = min_pair(min_pair(w.x, w.y, T()), min_pair(w.z, w.w, T()), T());
    const uint32_t b = min_pair(min_pair(w.x ^ kSigns, w.y ^ kSigns, T()), min_pair(w.z ^ kSigns, w.w ^ kSigns, T()), T());
    // least values of the even and the odd features, then the negated greatest ones
    uint32_t m = min_pair(__byte_perm(a, b, 0x5410), __byte_perm(a, b, 0x7632), T());
#pragma unroll
    for (int o = 1; o < D / 32; o <<= 1) m = min_pair(m, __shfl_xor_sync(0xffffffffu, m, o), T());
    float f[8];
    unpack16_t<T>(make_uint4(m, 0u, 0u, 0u), f);
    lo = f[0];
    hi = -f[1];
  }
}

template <typename T, int D>
MGQA_DEV Q4Piece quantise(const Eight<T> &e) {
  float x[8], lo, hi;
  e.values(x);
  extremes<T, D>(e, x, lo, hi);
  uint32_t least = __half_as_ushort(__float2half_rn(fminf(fmaxf(lo, -65504.f), 65504.f)));
  if (least == 0x8000u) least = 0u;
  const float base = __half2float(__ushort_as_half((unsigned short)least));
  const float range = __fmul_rn(__fsub_rn(hi, base), 1.f / 15.f);
  const __half scale = __float2half_rn(fminf(fmaxf(range, 0.f), 65504.f));
  const float step = __half2float(scale);
  const float inv = step > 0.f ? __frcp_rn(step) : 0.f;
  Q4Piece r;
  r.par = (uint32_t)__half_as_ushort(scale) | least << 16;
  // The quotients by the reciprocal and one correction, rounded as a division's (P.
  // Markstein, IBM J. Res. Develop. 34, 1990: the reciprocal is a rounded one, the
  // remainder exact); adding 1.5 2^23 rounds them to whole numbers, half to even, in
  // the low bits. Where least's rounding leaves values far outside the codes, and they
  // have to be clamped, the division does.
  uint32_t codes = 0u;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float d = __fsub_rn(x[i], base), q = __fmul_rn(d, inv);
    const float t = __fadd_rn(__fmaf_rn(__fmaf_rn(-q, step, d), inv, q), 12582912.f);
    codes += __float_as_uint(t) << (4 * i);
  }
  codes -= 0x4b400000u * 0x11111111u;
  if (!(__fmul_rn(__fsub_rn(lo, base), inv) > -0.499f && __fmul_rn(__fsub_rn(hi, base), inv) < 15.499f)) {
    codes = 0u;
#pragma unroll 1
    for (int i = 0; i < 8; ++i) {
      float u = x[0];
#pragma unroll
      for (int k = 1; k < 8; ++k) u = i == k ? x[k] : u;
      u = step > 0.f ? rintf(__fdiv_rn(__fsub_rn(u, base), step)) : 0.f;
      codes |= (uint32_t)(int)fminf(fmaxf(u, 0.f), 15.f) << (4 * i);
    }
  }
  if constexpr (D == 64) {
    // the bytes of groups 0 and 1 (2 and 3) by turns: the first group's thread keeps
    // the first two bytes of each, the other one the last two
    __syncwarp();
    const uint32_t other = __shfl_xor_sync(0xffffffffu, codes, 2);
    codes = (threadIdx.x & 2) ? __byte_perm(other, codes, 0x7362) : __byte_perm(codes, other, 0x5140);
  }
  r.codes = codes;
  return r;
}

// The thread's part of a record (null: none): its codes, and from the row's first
// thread the parameters. (Whole warps.)
template <int D>
MGQA_DEV void store_record(char *rec, const Q4Piece &r, int piece) {
  constexpr int GL = D / 32;  // threads of a group
  uint32_t g[4];
  const int first = (int)(threadIdx.x & 31) - piece;
  __syncwarp();
#pragma unroll
  for (int i = 0; i < 4; ++i) g[i] = __shfl_sync(0xffffffffu, r.par, first + i * GL);
  if (!rec) return;
  // (D = 64: threads 0..3 of a chunk have its words 0, 2, 1, 3)
  const int word = D == 64 ? (piece & ~3) | (piece & 1) << 1 | (piece >> 1 & 1) : piece;
  __stcs(reinterpret_cast<uint32_t *>(rec) + word, r.codes);
  if (piece == 0)
    __stcs(reinterpret_cast<uint4 *>(rec + D / 2),
           make_uint4(__byte_perm(g[0], g[1], 0x5410), __byte_perm(g[2], g[3], 0x5410), __byte_perm(g[0], g[1], 0x7632),
                      __byte_perm(g[2], g[3], 0x7632)));
}

template <typename T, int D>
__global__ void __launch_bounds__(kAppendThreads)
append_q4_kernel(const __grid_constant__ Q4Params qp) {
  constexpr int LR = D / 8;  // threads of a row
  const AppendParams &p = qp.a;
  const Pool &c = p.c;
  const int b = blockIdx.y, layer = blockIdx.z;
  grid_dependency_wait();
  allow_dependents();
  const int64_t cap = c.table ? (int64_t)c.max_pages * c.page_size : c.page_size;
  const auto load = [&](const int32_t *x) { return p.ints_apart ? __ldg(x) : __ldcg(x); };
  const int n = load(c.kv_len + b);
  const int cnt = p.count ? load(p.count + b) : p.T;
  const bool bad = n < 0 || cnt < 0 || cnt > p.T || (int64_t)n + cnt > cap;
  const int live = bad ? 0 : cnt;
  const int t0 = (int)blockIdx.x * p.block_rows, rows = max(0, min(p.block_rows, live - t0)) * c.Hkv;
  const int piece = threadIdx.x % LR;
  const auto pieces = [&](const uint32_t (&st)[4], int x, int y, int z) {  // of layer `layer`
    return (uint64_t)(uint32_t)layer * st[0] + (uint64_t)(uint32_t)x * st[1] + (uint64_t)(uint32_t)y * st[2] +
           (uint64_t)(uint32_t)z * st[3];
  };
  for (int r0 = 0; r0 < rows; r0 += (int)blockDim.x / LR) {  // (whole warps)
    const int r = r0 + (int)threadIdx.x / LR;
    const int tl = c.Hkv == 1 ? r : (int)__umulhi((uint32_t)r, qp.by_heads), h = r - tl * c.Hkv, t = t0 + tl;
    const bool mine = r < rows;
    int from = t;
    if (p.index && mine) from = load(p.index + (int64_t)b * p.T + t);
    const bool has = mine && (unsigned)from < (unsigned)p.T;
    Eight<T> kx{}, vx{};
    if (has) {
      const uint64_t at = pieces(qp.knstep, b, h, from), av = qp.alike ? at : pieces(qp.vnstep, b, h, from);
      kx.load(p.kn + (at * 16 + piece * (8 * (int)sizeof(T))));
      vx.load(p.vn + (av * 16 + piece * (8 * (int)sizeof(T))));
    }
    int page = b, slot = n + t;
    if (c.table && mine) {
      const int pi = qp.page_shift >= 0 ? slot >> qp.page_shift : slot / c.page_size;
      page = valid_page(c, load(c.table + (int64_t)b * c.table_stride + pi));
      slot -= pi * c.page_size;
    }
    const bool to = has && page >= 0;
    if (mine && !to && layer == 0 && piece == 0 && h == 0) report_error(c.err, MGQA_ERR_INVALID_ARG);
    char *k = nullptr, *v = nullptr;
    if (to) {
      const uint64_t at = pieces(qp.kstep, page, h, slot), av = qp.alike ? at : pieces(qp.vstep, page, h, slot);
      k = c.k + at * 16;
      v = c.v + av * 16;
    }
    store_record<D>(k, quantise<T, D>(kx), piece);
    store_record<D>(v, quantise<T, D>(vx), piece);
  }
  if (blockIdx.x == 0 && layer == 0 && threadIdx.x == 0) {
    if (bad) report_error(c.err, MGQA_ERR_INVALID_ARG);
    p.kv_len_out[b] = bad ? n : n + cnt;
  }
}

// ---- copies of (parts of) pages --------------------------------------------------

// Slots [0, slots) of page a of one layer's K or V to page b, by `warps` warps
// of which this is `warp`: a warp, or several, per head's rows (per run of 16-
// byte pieces, the whole page when it has no gaps).
constexpr int kCopyU = 4;
MGQA_DEV void copy_slots(char *base, const int64_t *st, int64_t layer, int a, int b, int heads, int slots,
                         int page_size, int pieces, int warp, int warps) {
  const char *src = base + layer * st[0] + (int64_t)a * st[1];
  char *dst = base + layer * st[0] + (int64_t)b * st[1];
  const bool rows_run = st[3] == pieces * 16;
  int per = slots * pieces;  // pieces of a run
  if (rows_run && slots == page_size && st[2] == (int64_t)page_size * st[3] && (int64_t)per * heads <= kMaxPagePieces) {
    per *= heads;
    heads = 1;
  }
  const int wph = max(1, warps / heads), step = 32 * wph;  // warps of a run
  if (warp >= wph * heads) return;
  for (int h = warp / wph; h < heads; h += warps / wph) {
    const char *sh = src + h * st[2];
    char *dh = dst + h * st[2];
    const int first = (warp % wph) * 32 + (int)(threadIdx.x & 31);
    if (rows_run) {
      const uint4 *from = reinterpret_cast<const uint4 *>(sh);
      uint4 *to = reinterpret_cast<uint4 *>(dh);
      for (int i = first; i < per; i += step * kCopyU) {
        uint4 x[kCopyU];
#pragma unroll
        for (int u = 0; u < kCopyU; ++u)
          if (i + u * step < per) x[u] = __ldcs(from + i + u * step);
#pragma unroll
        for (int u = 0; u < kCopyU; ++u)
          if (i + u * step < per) __stcs(to + i + u * step, x[u]);
      }
    } else {
      for (int i = first; i < per; i += step * 2) {  // rows apart: two pieces in flight
        const int64_t at = (i / pieces) * st[3] + (i % pieces) * 16;
        const int i2 = i + step;
        const int64_t at2 = (i2 / pieces) * st[3] + (i2 % pieces) * 16;
        uint4 y;
        if (i2 < per) y = __ldcs(reinterpret_cast<const uint4 *>(sh + at2));
        const uint4 x = __ldcs(reinterpret_cast<const uint4 *>(sh + at));
        __stcs(reinterpret_cast<uint4 *>(dh + at), x);
        if (i2 < per) __stcs(reinterpret_cast<uint4 *>(dh + at2), y);
      }
    }
  }
}

// ---- block-wide prefix sums --------------------------------------------------------

constexpr int kPlanThreads = 1024;

// Exclusive prefix sum over the block's threads; *total receives the sum.
// scratch: 33 ints. Every thread takes part.
MGQA_DEV int block_prefix(int x, int *scratch, int *total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int inc = x;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int up = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += up;
  }
  if (lane == 31) scratch[warp] = inc;
  __syncthreads();
  if (warp == 0) {
    int w = lane < (int)(blockDim.x >> 5) ? scratch[lane] : 0;
    int wi = w;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int up = __shfl_up_sync(0xffffffffu, wi, o);
      if (lane >= o) wi += up;
    }
    scratch[lane] = wi - w;
    if (lane == 31) scratch[32] = wi;
  }
  __syncthreads();
  const int r = scratch[warp] + inc - x;
  *total = scratch[32];
  __syncthreads();
  return r;
}

// Bits of the pages [32 w, 32 w + 32) with ref > 0 (used) for every word of
// the pool, by whole warps.
MGQA_DEV void used_bitmap(const Pool &p, uint32_t *bits) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  const int W = (p.num_pages + 31) / 32;
  constexpr int U = 8;
  for (int w0 = warp; w0 < W; w0 += warps * U) {
    int r[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int page = (w0 + u * warps) * 32 + lane;
      r[u] = page < p.num_pages ? __ldcg(p.ref + page) : 0;
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const uint32_t b = __ballot_sync(0xffffffffu, r[u] > 0);
      if (lane == 0 && w0 + u * warps < W) bits[w0 + u * warps] = b;
    }
  }
}

// ---- fork ----------------------------------------------------------------------------

struct Pair {
  int32_t src, dst;   // dst -1: skipped
  int32_t len, full;  // the source's length, and its filled pages
  int32_t need;       // table entries wanted (-1: more than a row has)
  int32_t off;        // first of its pages in the list of fresh ones
  int32_t ok;
  int32_t copy;       // page whose filled slots are copied (-1: none)
};

// Entries of a staged row that keeps its request (src == dst), besides pages
// and -1: a fresh page, replacing nothing, or page e which the row gives back.
// (A row that takes over another's gets fresh pages from its `full` on.)
constexpr int32_t kFresh = -2;
MGQA_DEV int32_t fresh_for(int e) { return e < 0 ? kFresh : -3 - e; }

struct ForkParams {
  Pool c;
  int32_t n, extra;
  const int32_t *src, *dst;
  int32_t *stage;  // [n][max_pages]
  Pair *pairs;     // [n]
  int32_t *fresh;  // [num_pages]
};

constexpr int kForkThreads = 256;

// Pair i: its numbers, its source's row staged, pages given back and shares taken.
__global__ void __launch_bounds__(kForkThreads)
fork_gather_kernel(const __grid_constant__ ForkParams p) {
  const Pool &c = p.c;
  const int i = blockIdx.x, tid = threadIdx.x;
  grid_dependency_wait();
  allow_dependents();
  const int s = __ldg(p.src + i), d = __ldg(p.dst + i);
  bool taken = false;  // an earlier pair has this dst
  for (int k = tid; k < i; k += kForkThreads) taken = taken || __ldg(p.dst + k) == d;
  const bool skip = __syncthreads_or(taken) || d < 0 || d >= c.rows || s < -1 || s >= c.rows;
  int len = 0;
  const int64_t cap = (int64_t)c.max_pages * c.page_size;
  if (!skip && s >= 0) {
    len = __ldg(c.kv_len + s);
    if (len < 0 || len > cap) {
      if (tid == 0) report_error(c.err, MGQA_ERR_INVALID_ARG);
      len = len < 0 ? 0 : (int)cap;
    }
  }
  const int full = len / c.page_size;
  if (tid == 0) {
    if (skip) report_error(c.err, MGQA_ERR_INVALID_ARG);
    const int64_t need = s < 0 ? 0 : ((int64_t)len + p.extra + c.page_size - 1) / c.page_size;
    p.pairs[i] = Pair{s, skip ? -1 : d, len, full, need > c.max_pages ? -1 : (int32_t)need, 0, 0, -1};
  }
  if (skip) return;
  for (int j = tid; j < c.max_pages; j += kForkThreads) {
    const int e = s >= 0 ? valid_page(c, __ldg(c.table + (int64_t)s * c.table_stride + j)) : -1;
    p.stage[(int64_t)i * c.max_pages + j] = e;
    if (s != d) {
      const int held = valid_page(c, __ldg(c.table + (int64_t)d * c.table_stride + j));
      if (held >= 0) atomicSub(c.ref + held, 1);
      if (e >= 0 && j < full) atomicAdd(c.ref + e, 1);
    }
  }
}

// dynamic shared memory: the bitmap of free pages
__global__ void __launch_bounds__(kPlanThreads)
fork_plan_kernel(const __grid_constant__ ForkParams p) {
  extern __shared__ uint32_t bits[];
  __shared__ int scratch[33], req_s[kMaxForks];
  const Pool &c = p.c;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int W = (c.num_pages + 31) / 32;
  grid_dependency_wait();
  allow_dependents();
  used_bitmap(c, bits);
  __syncthreads();
  for (int w = tid; w < W; w += kPlanThreads)
    bits[w] = ~bits[w] & low_mask(c.num_pages - 32 * w);
  __syncthreads();
  // Requests. A row taken over asks for its pages from `full` on; a kept row for
  // those it lacks or shares, noted in its staged row. The pages that copies read
  // are not handed out.
  Pair pr{-1, -1, 0, 0, 0, 0, 0, -1};
  int req = 0;
  if (tid < p.n) {
    const int4 *q = reinterpret_cast<const int4 *>(p.pairs + tid);
    const int4 a = __ldcg(q), b = __ldcg(q + 1);
    pr = Pair{a.x, a.y, a.z, a.w, b.x, 0, 0, -1};
  }
  auto copy_from = [&](int i, int e) {  // the filled slots of page e go to a fresh one
    if (e >= 0) atomicAnd(&bits[e >> 5], ~(1u << (e & 31)));
    else report_error(c.err, MGQA_ERR_INVALID_ARG);  // the source lacks its last page
    p.pairs[i].copy = e;
  };
  const bool asks = pr.dst >= 0 && pr.src >= 0 && pr.need >= 0;
  constexpr int kFew = 8;  // entries that one thread looks at
  if (asks && pr.src != pr.dst) {
    req = pr.need - pr.full;
    if (pr.len % c.page_size) copy_from(tid, __ldcg(p.stage + (int64_t)tid * c.max_pages + pr.full));
  } else if (asks && pr.need - pr.full <= kFew) {
    int32_t *row = p.stage + (int64_t)tid * c.max_pages + pr.full;
    int e[kFew], r[kFew];
#pragma unroll
    for (int k = 0; k < kFew; ++k) e[k] = k < pr.need - pr.full ? __ldcg(row + k) : -1;
#pragma unroll
    for (int k = 0; k < kFew; ++k) r[k] = e[k] >= 0 ? __ldcg(c.ref + e[k]) : 2;
#pragma unroll
    for (int k = 0; k < kFew; ++k)
      if (k < pr.need - pr.full && r[k] > 1) {
        if (k == 0 && pr.len % c.page_size) copy_from(tid, e[0]);
        row[k] = fresh_for(e[k]);
        ++req;
      }
  } else if (asks) {
    req = -1;
  }
  if (tid < p.n) req_s[tid] = req;
  __syncthreads();
  for (int i = warp; i < p.n; i += kPlanThreads / 32) {  // kept rows with many entries: a warp each
    if (req_s[i] >= 0) continue;
    const int full = __ldcg(&p.pairs[i].full), need = __ldcg(&p.pairs[i].need), len = __ldcg(&p.pairs[i].len);
    int32_t *row = p.stage + (int64_t)i * c.max_pages;
    int n = 0;
    for (int j0 = full; j0 < need; j0 += 32) {
      const int j = j0 + lane;
      bool fresh = false;
      if (j < need) {
        const int e = __ldcg(row + j);
        fresh = e < 0 || __ldcg(c.ref + e) > 1;
        if (fresh) {
          if (j == full && len % c.page_size) copy_from(i, e);
          row[j] = fresh_for(e);
        }
      }
      n += __popc(__ballot_sync(0xffffffffu, fresh));
    }
    __syncwarp();
    if (lane == 0) req_s[i] = n;
  }
  __syncthreads();
  // A pair that wants more pages than there are is not served, whatever it wants: its
  // request counts as one more than that, so that all of them add up within 32 bits
  // (uncut, 128 rows of 2^24 entries would not).
  static_assert((int64_t)kMaxForks * (kMaxPages + 1) < 0x7fffffff, "the requests' sum");
  if (tid < p.n) req = min(req_s[tid], c.num_pages + 1);
  // the free pages: every thread owns a run of words
  const int per = (W + kPlanThreads - 1) / kPlanThreads;
  int mine = 0, avail = 0, total = 0;
  for (int w = tid * per; w < min(W, tid * per + per); ++w) mine += __popc(bits[w]);
  int at = block_prefix(mine, scratch, &avail);
  const int off = block_prefix(tid < p.n ? req : 0, scratch, &total);
  bool ok = false;
  if (tid < p.n) {
    ok = pr.dst >= 0 && pr.need >= 0 && (req == 0 || off + req <= avail);
    if (pr.dst >= 0 && !ok) report_error(c.err, MGQA_ERR_INVALID_ARG);
    p.pairs[tid].off = off;
    p.pairs[tid].ok = ok;
  }
  // pages handed out: those of the pairs that succeed, which come first
  int given;
  block_prefix(ok ? req : 0, scratch, &given);
  for (int w = tid * per; w < min(W, tid * per + per) && at < given; ++w)
    for (uint32_t x = bits[w]; x && at < given; x &= x - 1, ++at) {
      const int page = 32 * w + __ffs(x) - 1;
      p.fresh[at] = page;
      c.ref[page] = 1;
    }
}

// grid (pair, layer, K or V)
__global__ void __launch_bounds__(kForkThreads)
fork_apply_kernel(const __grid_constant__ ForkParams p) {
  const Pool &c = p.c;
  const int i = blockIdx.x, layer = blockIdx.y, tid = threadIdx.x, lane = tid & 31;
  grid_dependency_wait();
  allow_dependents();
  const int4 *q = reinterpret_cast<const int4 *>(p.pairs + i);
  const int4 qa = q[0], qb = q[1];
  const Pair pr{qa.x, qa.y, qa.z, qa.w, qb.x, qb.y, qb.z, qb.w};
  if (pr.dst < 0) return;
  if (layer == 0 && blockIdx.z == 0) {
    int32_t *row = c.table + (int64_t)pr.dst * c.table_stride;
    const int32_t *from = p.stage + (int64_t)i * c.max_pages;
    if (!pr.ok) {
      if (pr.src != pr.dst) {  // the shares go back and the row is empty
        for (int j = tid; j < c.max_pages; j += kForkThreads) {
          const int e = from[j];
          if (j < pr.full && e >= 0) atomicSub(c.ref + e, 1);
          row[j] = -1;
        }
        if (tid == 0) c.kv_len[pr.dst] = 0;
      }
    } else {
      if (tid == 0) c.kv_len[pr.dst] = pr.len;
      const bool keep = pr.src == pr.dst;
      for (int j = tid; j < c.max_pages; j += kForkThreads)
        if (j < pr.full) row[j] = from[j];
        else if (j >= max(pr.full, pr.need)) row[j] = keep ? from[j] : -1;
      if (tid < 32) {  // the entries that got fresh pages, in order
        int at = pr.off;
        for (int j0 = pr.full; j0 < pr.need; j0 += 32) {
          const int j = j0 + lane;
          const int e = j < pr.need ? from[j] : -1;
          const bool fresh = j < pr.need && (!keep || e <= kFresh);
          const uint32_t m = __ballot_sync(0xffffffffu, fresh);
          if (fresh) {
            row[j] = p.fresh[at + __popc(m & ((1u << lane) - 1u))];
            if (keep && e < kFresh) atomicSub(c.ref + (-3 - e), 1);
          } else if (j < pr.need) {
            row[j] = e;
          }
          at += __popc(m);
        }
      }
    }
  }
  if (!pr.ok || pr.copy < 0) return;
  const int to = p.fresh[pr.off];  // the copied entry is the pair's first fresh one
  copy_slots(blockIdx.z ? c.v : c.k, blockIdx.z ? c.vs : c.ks, layer, pr.copy, to, c.Hkv, pr.len % c.page_size,
             c.page_size, c.pieces, tid / 32, kForkThreads / 32);
}

// ---- compact ---------------------------------------------------------------------------

struct CompactParams {
  Pool c;
  int32_t *table_out;
  int64_t table_out_stride;
  int32_t *ref_out, *used_out;
  int32_t *state;           // [0]: used pages U, [1]: moves
  int32_t *from, *to;       // [num_pages / 2 + 1] moves
  uint32_t *bits;           // used pages
  int32_t *rank;            // [words] moves ahead of each word
  int32_t warp_segments;    // a warp per segment instead of a block
};

__global__ void __launch_bounds__(kPlanThreads)
compact_plan_kernel(const __grid_constant__ CompactParams p) {
  extern __shared__ uint32_t bits[];
  __shared__ int scratch[33];
  const Pool &c = p.c;
  const int tid = threadIdx.x;
  const int W = (c.num_pages + 31) / 32, per = (W + kPlanThreads - 1) / kPlanThreads;
  grid_dependency_wait();
  allow_dependents();
  used_bitmap(c, bits);
  __syncthreads();
  int used = 0, moves = 0, holes = 0, n = 0;
  const int w0 = tid * per, w1 = min(W, w0 + per);
  for (int w = w0; w < w1; ++w) n += __popc(bits[w]);
  block_prefix(n, scratch, &used);
  auto moving = [&](int w) { return bits[w] & ~low_mask(used - 32 * w); };
  auto hole = [&](int w) { return ~bits[w] & low_mask(used - 32 * w); };
  int m = 0, h = 0;
  for (int w = w0; w < w1; ++w) {
    m += __popc(moving(w));
    h += __popc(hole(w));
  }
  int mi = block_prefix(m, scratch, &moves), hi = block_prefix(h, scratch, &holes);
  for (int w = w0; w < w1; ++w) {
    p.rank[w] = mi;
    p.bits[w] = bits[w];
    for (uint32_t x = moving(w); x; x &= x - 1) p.from[mi++] = 32 * w + __ffs(x) - 1;
    for (uint32_t x = hole(w); x; x &= x - 1) p.to[hi++] = 32 * w + __ffs(x) - 1;
  }
  if (tid == 0) {
    p.state[0] = used;
    p.state[1] = moves;
    if (p.used_out) *p.used_out = used;
  }
}

constexpr int kCompactThreads = 256;

__global__ void __launch_bounds__(kCompactThreads)
compact_apply_kernel(const __grid_constant__ CompactParams p) {
  const Pool &c = p.c;
  const int tid = threadIdx.x;
  grid_dependency_wait();
  allow_dependents();
  const int used = p.state[0], moves = p.state[1];
  // the copies: a segment is one (move, layer, K or V)
  const int64_t both = (int64_t)c.layers * 2, segs = moves * both;
  const int group = p.warp_segments ? 32 : kCompactThreads;
  const int64_t step = (int64_t)gridDim.x * (kCompactThreads / group);
  for (int64_t s = (int64_t)blockIdx.x * (kCompactThreads / group) + tid / group; s < segs; s += step) {
    const int64_t r = s % both;
    const int mv = (int)(s / both);
    copy_slots((r & 1) ? c.v : c.k, (r & 1) ? c.vs : c.ks, r >> 1, p.from[mv], p.to[mv], c.Hkv, c.page_size,
               c.page_size, c.pieces, tid % group / 32, group / 32);
  }
  // the renamed table and the counts; a count is read and written by one thread only
  const int64_t t0 = (int64_t)blockIdx.x * kCompactThreads + tid, ts = (int64_t)gridDim.x * kCompactThreads;
  auto word_rank = [&](int page) {
    const int w = page >> 5;
    return p.rank[w] + __popc(p.bits[w] & ~low_mask(used - 32 * w) & low_mask(page & 31));
  };
  for (int64_t u = t0; u < (int64_t)c.rows * c.max_pages; u += ts) {
    const int r = (int)(u / c.max_pages), j = (int)(u % c.max_pages);
    int e = __ldcg(c.table + (int64_t)r * c.table_stride + j);  // (past the L1, as append's lengths when they share a line)
    if (e >= c.num_pages || e < -1) {
      report_error(c.err, MGQA_ERR_INVALID_ARG);
      e = -1;
    }
    if (e >= used) {  // (an entry that names a free page keeps its name)
      const bool in_use = (p.bits[e >> 5] >> (e & 31)) & 1u;
      if (in_use) e = p.to[word_rank(e)];
    }
    p.table_out[(int64_t)r * p.table_out_stride + j] = e;
  }
  for (int64_t k = t0; k < moves; k += ts) {
    const int a = p.from[k], b = p.to[k], r = __ldcg(c.ref + a);
    p.ref_out[b] = r;
    p.ref_out[a] = 0;
  }
  if (p.ref_out != c.ref)
    for (int64_t u = t0; u < c.num_pages; u += ts) {
      const int page = (int)u;
      const bool in_use = (p.bits[page >> 5] >> (page & 31)) & 1u;
      if (in_use == (page < used)) p.ref_out[page] = __ldcg(c.ref + page);
    }
}

int64_t aligned16(int64_t n) { return (n + 15) & ~(int64_t)15; }

mgqa_status launched(cudaError_t e, const char *what) {
  if (e != cudaSuccess) return fail(MGQA_ERR_CUDA, "%s launch: %s", what, cudaGetErrorString(e));
  return MGQA_OK;
}

}  // namespace

size_t cache_pages_workspace_bytes(const mgqa_cache &c, int n) {
  const int64_t words = (c.num_pages + 31) / 32;
  const int64_t fork = aligned16((int64_t)n * c.max_pages * 4) + aligned16((int64_t)n * (int64_t)sizeof(Pair)) +
                       aligned16((int64_t)c.num_pages * 4);
  const int64_t compact = 16 + 2 * aligned16(((int64_t)c.num_pages / 2 + 1) * 4) + 2 * aligned16(words * 4);
  return (size_t)std::max(n ? fork : 0, compact);
}

mgqa_status launch_cache_append(const mgqa_cache &c, const void *k_new, const void *v_new, const int64_t *ks,
                                const int64_t *vs, int32_t T, const int32_t *index, const int32_t *count,
                                int32_t *kv_len_out, bool q4, cudaStream_t s) {
  AppendParams p{};
  p.c = pool_of(c);
  if (q4) {
    p.c.pieces = c.D / 8;  // threads of a row
    for (int t = 0; t < 4; ++t) {
      p.c.ks[t] = c.k_stride[t];
      p.c.vs[t] = c.v_stride[t];
    }
  }
  p.kn = static_cast<const char *>(k_new);
  p.vn = static_cast<const char *>(v_new);
  const int64_t es = c.dtype == MGQA_FP32 ? 4 : 2;
  for (int t = 0; t < 4; ++t) {
    p.kns[t] = ks[t] * es;
    p.vns[t] = vs[t] * es;
  }
  p.T = T; p.index = index; p.count = count; p.kv_len_out = kv_len_out;
  const auto apart = [&](const int32_t *x, int64_t n) {  // no line of x[0, n) holds a new length
    const uintptr_t line = 128, in = reinterpret_cast<uintptr_t>(x), to = reinterpret_cast<uintptr_t>(kv_len_out);
    return !x || (in + 4 * (uintptr_t)n - 1) / line < to / line || (to + 4 * (uintptr_t)c.rows - 1) / line < in / line;
  };
  p.ints_apart = apart(c.kv_len, c.rows) && apart(count, c.rows) && apart(index, (int64_t)c.rows * T) &&
                 apart(c.page_table, (int64_t)(c.rows - 1) * c.table_stride + c.max_pages);
  const int64_t per = (int64_t)c.Hkv * p.c.pieces;
  if (per > (1 << 20)) return fail(MGQA_ERR_UNSUPPORTED, "cache append: rows of more than 16 MB");
  p.block_rows = (int32_t)std::max<int64_t>(1, kAppendThreads / per);
  // (four rounds a block: 32768 rows of 8 x 128 55.7 us, one 59.6, eight 58.0)
  if (q4 && per <= kAppendThreads) p.block_rows = std::min(T, p.block_rows * 4);
  const int64_t bx = (T + p.block_rows - 1) / p.block_rows;
  if (c.rows > 65535 || c.layers > 65535 || bx > 0x7fffffff)
    return fail(MGQA_ERR_UNSUPPORTED, "more than 65535 requests or layers");
  const dim3 grid((unsigned)bx, c.rows, c.layers);
  if (!q4) return launched(launch_pdl(append_kernel, grid, dim3(kAppendThreads), 0, s, p), "cache append");
  Q4Params qp{};
  bool fits = c.Hkv <= 1 << 15;
  for (int t = 0; t < 4; ++t) {
    const int64_t st[4] = {p.c.ks[t] / 16, p.c.vs[t] / 16, p.kns[t] / 16, p.vns[t] / 16};
    for (const int64_t x : st) fits = fits && x <= 0xffffffffll;
    qp.kstep[t] = (uint32_t)st[0];
    qp.vstep[t] = (uint32_t)st[1];
    qp.knstep[t] = (uint32_t)st[2];
    qp.vnstep[t] = (uint32_t)st[3];
  }
  if (!fits) return fail(MGQA_ERR_UNSUPPORTED, "4-bit append: strides past 2^36 bytes, or more than 2^15 KV heads");
  qp.alike = std::equal(qp.kstep, qp.kstep + 4, qp.vstep) && std::equal(qp.knstep, qp.knstep + 4, qp.vnstep);
  qp.page_shift = -1;
  if ((c.page_size & (c.page_size - 1)) == 0)
    for (qp.page_shift = 0; (1 << qp.page_shift) < c.page_size;) ++qp.page_shift;
  qp.by_heads = (uint32_t)((((uint64_t)1 << 32) + c.Hkv - 1) / c.Hkv);
  qp.a = p;
  const auto kern = c.dtype == MGQA_BF16   ? (c.D == 64 ? append_q4_kernel<__nv_bfloat16, 64> : append_q4_kernel<__nv_bfloat16, 128>)
                    : c.dtype == MGQA_FP16 ? (c.D == 64 ? append_q4_kernel<__half, 64> : append_q4_kernel<__half, 128>)
                                           : (c.D == 64 ? append_q4_kernel<float, 64> : append_q4_kernel<float, 128>);
  // (no idle threads where a request has few rows: a token of 32 requests x 32 layers, 8 heads
  // of 128, in one wave of blocks)
  const int threads = (int)std::min<int64_t>(kAppendThreads, (p.block_rows * per + 31) / 32 * 32);
  return launched(launch_pdl(kern, grid, dim3(threads), 0, s, qp), "cache append");
}

mgqa_status launch_cache_fork(const mgqa_cache &c, int n, const int32_t *src, const int32_t *dst, int32_t extra,
                              void *ws, cudaStream_t s) {
  if (c.layers > 65535) return fail(MGQA_ERR_UNSUPPORTED, "more than 65535 layers");
  ForkParams p{};
  p.c = pool_of(c);
  p.n = n; p.extra = extra; p.src = src; p.dst = dst;
  char *w = static_cast<char *>(ws);
  p.stage = reinterpret_cast<int32_t *>(w);
  w += aligned16((int64_t)n * c.max_pages * 4);
  p.pairs = reinterpret_cast<Pair *>(w);
  w += aligned16((int64_t)n * (int64_t)sizeof(Pair));
  p.fresh = reinterpret_cast<int32_t *>(w);
  const int smem = (c.num_pages + 31) / 32 * 4;
  static std::atomic<uint64_t> attr{0};
  mgqa_status st = ensure_smem_attr(fork_plan_kernel, kMaxPages / 8, attr, "fork planning kernel");
  if (st != MGQA_OK) return st;
  st = launched(launch_pdl(fork_gather_kernel, dim3(n), dim3(kForkThreads), 0, s, p), "cache fork");
  if (st != MGQA_OK) return st;
  st = launched(launch_pdl(fork_plan_kernel, dim3(1), dim3(kPlanThreads), smem, s, p), "cache fork");
  if (st != MGQA_OK) return st;
  return launched(launch_pdl(fork_apply_kernel, dim3(n, c.layers, 2), dim3(kForkThreads), 0, s, p), "cache fork");
}

mgqa_status launch_cache_compact(const mgqa_cache &c, int32_t *table_out, int64_t table_out_stride, int32_t *ref_out,
                                 int32_t *used_out, void *ws, cudaStream_t s) {
  CompactParams p{};
  p.c = pool_of(c);
  p.table_out = table_out; p.table_out_stride = table_out_stride;
  p.ref_out = ref_out; p.used_out = used_out;
  const int64_t words = (c.num_pages + 31) / 32;
  char *w = static_cast<char *>(ws);
  p.state = reinterpret_cast<int32_t *>(w);
  w += 16;
  p.from = reinterpret_cast<int32_t *>(w);
  w += aligned16(((int64_t)c.num_pages / 2 + 1) * 4);
  p.to = reinterpret_cast<int32_t *>(w);
  w += aligned16(((int64_t)c.num_pages / 2 + 1) * 4);
  p.bits = reinterpret_cast<uint32_t *>(w);
  w += aligned16(words * 4);
  p.rank = reinterpret_cast<int32_t *>(w);
  const int64_t seg = (int64_t)c.Hkv * c.page_size * p.c.pieces;  // 16-byte pieces of a segment
  p.warp_segments = seg <= 256;
  static std::atomic<uint64_t> attr{0};
  mgqa_status st = ensure_smem_attr(compact_plan_kernel, kMaxPages / 8, attr, "compact planning kernel");
  if (st != MGQA_OK) return st;
  const int sms = device_sm_count();
  if (sms < 1) return fail(MGQA_ERR_CUDA, "cannot read the SM count of the current device");
  st = launched(launch_pdl(compact_plan_kernel, dim3(1), dim3(kPlanThreads), (size_t)words * 4, s, p),
                "cache compaction");
  if (st != MGQA_OK) return st;
  // at most half the pool moves
  const int64_t segs = ((int64_t)c.num_pages / 2 + 1) * c.layers * 2 / (p.warp_segments ? kCompactThreads / 32 : 1) + 1;
  const int64_t meta = ((int64_t)c.rows * c.max_pages + c.num_pages) / kCompactThreads + 1;
  const int grid = (int)std::min<int64_t>((int64_t)sms * 8, std::max(segs, meta));
  return launched(launch_pdl(compact_apply_kernel, dim3(grid), dim3(kCompactThreads), 0, s, p), "cache compaction");
}

}  // namespace mgqa
