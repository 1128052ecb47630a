// Register-tiled fp32 products of the CUDA-core attention kernels: 64 keys per
// tile, K and V in shared memory as TMA leaves them (boxes of 64 rows x 32
// floats, 128-byte swizzled), 256 threads over ROWS = 32, 48 or 64 query rows.
//
// A multiply-add reads its operands from registers, so the shared-memory reads
// per product fall with a thread's tile, which is as large as the registers
// allow: the threads are two groups of 8 x 16, each over half of the head dim in
// the scores and half of the keys in the values, and a thread (ty, tx) has rows
// ty + 8 a (a < ROWS / 8) by keys tx + 16 c, then the same rows by features
// 4 tx + 64 c .. + 3. Each group owns half of a thread's rows: it adds the other
// group's part of their scores, runs their softmax and writes them out. Products
// are packed pairs of fp32 multiply-adds (one instruction for two).
// At 64 rows and D = 128 a tile then needs 8192 cycles of multiply-adds and about
// as many of shared-memory reads; it takes about twice that (47 % of the fp32
// rate on 4096 queries x 16 heads, window 4096: 1854 us), since eight warps, all
// an SM's registers, do not cover one another's latencies. One group with tiles
// of 4 x 4 and no block barrier: 16 trees of 24 drafts over 8192 slots 1387 us
// against 1270 (in blocks of 64 rows), of 6 drafts 435 against 343, that prefill
// 1820.
#pragma once

#include "common.cuh"
#include "tc_ptx.cuh"

namespace mgqa {
namespace simt {

constexpr int kBox = 64 * 128;  // bytes of a box
constexpr int kXP = 80;         // row pitch of scores and weights (floats): two rows of a warp in different banks
constexpr int kThreads = 256;

// The two groups' common buffers. Alternating tiles use alternating halves, so a
// tile's writes need no barrier against the previous tile's reads.
template <int ROWS, int D>
struct Shared {
  union {
    float x[2][ROWS][kXP];  // parts of the scores, then the weights in their place
    float o[ROWS][D];       // after the last tile: the other group's rows
  };
  float f[2][ROWS];         // factors for what was summed before the tile
};

MGQA_DEV void lds_pairs(uint64_t &a, uint64_t &b, const void *p) {  // 16 bytes as two pairs
  asm volatile("ld.shared.v2.u64 {%0, %1}, [%2];" : "=l"(a), "=l"(b) : "r"(smem_u32(p)));
}
MGQA_DEV float pair_sum(uint64_t x) {
  float a, b;
  tc::upk2(x, a, b);
  return a + b;
}
MGQA_DEV uint64_t mul2(uint64_t a, float f) {
  uint64_t d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(tc::pk2(f, f)));
  return d;
}

// A thread's place: group h, and which rows of the block it owns.
struct Place {
  int tx, ty, h;
  MGQA_DEV explicit Place(int tid) : tx(tid & 15), ty((tid >> 4) & 7), h(tid >> 7) {}
  template <int RPG> MGQA_DEV int own(int a) const { return ty + 8 * (h * (RPG / 2) + a); }
  template <int RPG> MGQA_DEV int others(int a) const { return ty + 8 * ((1 - h) * (RPG / 2) + a); }
};

// s[a][c] = <q row ty + 8 a, key tx + 16 c> over group h's half of the head dim.
// QP: row pitch of q (floats).
template <int D, int RPG, int QP>
MGQA_DEV void scores(float (&s)[RPG][4], const float *q, const unsigned char *kt, const Place &at) {
  uint64_t acc[RPG][4];
#pragma unroll
  for (int a = 0; a < RPG; ++a)
#pragma unroll
    for (int c = 0; c < 4; ++c) acc[a][c] = 0ull;
  const unsigned char *krow = kt + at.h * (D / 64) * kBox + at.tx * 128;
  const float *qrow = q + at.ty * QP + at.h * (D / 2);
#pragma unroll
  for (int b = 0; b < D / 64; ++b)
#pragma unroll 4
    for (int d4 = 0; d4 < 8; ++d4) {
      uint64_t k0[4], k1[4];
      const int off = b * kBox + ((d4 ^ (at.tx & 7)) << 4);
#pragma unroll
      for (int c = 0; c < 4; ++c) lds_pairs(k0[c], k1[c], krow + off + c * (16 * 128));
#pragma unroll
      for (int a = 0; a < RPG; ++a) {
        uint64_t q0, q1;
        lds_pairs(q0, q1, qrow + 8 * a * QP + b * 32 + d4 * 4);
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          acc[a][c] = tc::fma2(q0, k0[c], acc[a][c]);
          acc[a][c] = tc::fma2(q1, k1[c], acc[a][c]);
        }
      }
    }
#pragma unroll
  for (int a = 0; a < RPG; ++a)
#pragma unroll
    for (int c = 0; c < 4; ++c) s[a][c] = pair_sum(acc[a][c]);
}

// o[a][c] (features 4 tx + 64 c .. + 3 of row ty + 8 a, as two pairs) += weights
// times V over group h's half of the keys. ok: which of those count (the rows of
// the others may hold anything).
template <int D, int RPG>
MGQA_DEV void values(uint64_t (&o)[RPG][D / 64][2], const float *w, const unsigned char *vt, const Place &at,
                     uint32_t ok) {
  const float *wrow = w + at.ty * kXP + 32 * at.h;
  const unsigned char *vbox = vt + (at.tx >> 3) * kBox + 32 * at.h * 128;
#pragma unroll 2
  for (int k = 0; k < 32; k += 4) {
    float4 w4[RPG];
#pragma unroll
    for (int a = 0; a < RPG; ++a) w4[a] = *reinterpret_cast<const float4 *>(wrow + 8 * a * kXP + k);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      uint64_t v[D / 64][2];
      const unsigned char *vr = vbox + (k + e) * 128 + (((at.tx & 7) ^ ((k + e) & 7)) << 4);
#pragma unroll
      for (int c = 0; c < D / 64; ++c) lds_pairs(v[c][0], v[c][1], vr + c * 2 * kBox);
      if (ok != 0xffffffffu && !((ok >> (k + e)) & 1u))
#pragma unroll
        for (int c = 0; c < D / 64; ++c) v[c][0] = v[c][1] = 0ull;
#pragma unroll
      for (int a = 0; a < RPG; ++a) {
        const float we = e == 0 ? w4[a].x : e == 1 ? w4[a].y : e == 2 ? w4[a].z : w4[a].w;
        const uint64_t w2 = tc::pk2(we, we);
#pragma unroll
        for (int c = 0; c < D / 64; ++c) {
          o[a][c][0] = tc::fma2(w2, v[c][0], o[a][c][0]);
          o[a][c][1] = tc::fma2(w2, v[c][1], o[a][c][1]);
        }
      }
    }
  }
}

// One row of the running softmax over a tile's scores, held by the 16 threads
// of a half-warp (4 keys each, in log2 units, masked ones -inf): the weights go
// to w, the factor for what was summed before is returned.
MGQA_DEV float softmax_row(const float (&s)[4], float &m, float &l, float *w, int tx) {
  float mx = fmaxf(m, fmaxf(fmaxf(s[0], s[1]), fmaxf(s[2], s[3])));
#pragma unroll
  for (int off = 1; off < 16; off <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, off));
  const float mb = mx == -INFINITY ? 0.f : mx;  // nothing seen yet: every weight is 0
  const float f = exp2f(m - mb);
  m = mx;
  l *= f;
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    const float x = exp2f(s[c] - mb);
    l += x;
    w[tx + 16 * c] = x;
  }
  return f;
}

// One tile for the block's 256 threads. m, l: of the thread's own rows; see(a, col,
// score): own row a's score at key col in log2 units, -inf where it is masked.
// `it` alternates between 0 and 1; without `ok` only the barriers are kept.
template <int D, int RPG, int QP, typename See>
MGQA_DEV void tile(bool ok, int it, const float *q, const unsigned char *kt, const unsigned char *vt,
                   Shared<8 * RPG, D> &sh, uint64_t (&o)[RPG][D / 64][2], float (&m)[RPG / 2], float (&l)[RPG / 2],
                   const Place &at, uint32_t ok_lo, uint32_t ok_hi, See see) {
  constexpr int H = RPG / 2;
  float *x = &sh.x[it][0][0], *fs = sh.f[it];
  float s[RPG][4];
#pragma unroll
  for (int a = 0; a < RPG; ++a) s[a][0] = s[a][1] = s[a][2] = s[a][3] = 0.f;
  if (ok) scores<D, RPG, QP>(s, q, kt, at);
#pragma unroll
  for (int a = 0; a < H; ++a)
#pragma unroll
    for (int c = 0; c < 4; ++c) x[at.others<RPG>(a) * kXP + at.tx + 16 * c] = at.h ? s[a][c] : s[H + a][c];
  named_sync(1, kThreads);
#pragma unroll
  for (int a = 0; a < H; ++a) {
    float *row = x + at.own<RPG>(a) * kXP;
    float v[4];
#pragma unroll
    for (int c = 0; c < 4; ++c)
      v[c] = see(a, at.tx + 16 * c, (at.h ? s[H + a][c] : s[a][c]) + row[at.tx + 16 * c]);
    const float f = softmax_row(v, m[a], l[a], row, at.tx);
    if (at.tx == 0) fs[at.own<RPG>(a)] = f;
  }
  named_sync(1, kThreads);
  if (!ok) return;
#pragma unroll
  for (int a = 0; a < RPG; ++a) {
    const float f = fs[at.ty + 8 * a];
#pragma unroll
    for (int c = 0; c < D / 64; ++c) {
      o[a][c][0] = mul2(o[a][c][0], f);
      o[a][c][1] = mul2(o[a][c][1], f);
    }
  }
  values<D, RPG>(o, x, vt, at, at.h ? ok_hi : ok_lo);
}

// After the last tile: x[a] gets the thread's own rows with both groups' keys,
// l[a] their sums.
template <int D, int RPG>
MGQA_DEV void finish(Shared<8 * RPG, D> &sh, const uint64_t (&o)[RPG][D / 64][2], float (&l)[RPG / 2],
                     float (&x)[RPG / 2][D / 64][4], const Place &at) {
  constexpr int H = RPG / 2;
  named_sync(1, kThreads);  // every weight has been read
#pragma unroll
  for (int a = 0; a < H; ++a)
#pragma unroll
    for (int c = 0; c < D / 64; ++c) {
      float y[4];
      tc::upk2(at.h ? o[a][c][0] : o[H + a][c][0], y[0], y[1]);
      tc::upk2(at.h ? o[a][c][1] : o[H + a][c][1], y[2], y[3]);
      *reinterpret_cast<float4 *>(&sh.o[at.others<RPG>(a)][at.tx * 4 + 64 * c]) = make_float4(y[0], y[1], y[2], y[3]);
    }
  named_sync(1, kThreads);
#pragma unroll
  for (int a = 0; a < H; ++a) {
#pragma unroll
    for (int off = 1; off < 16; off <<= 1) l[a] += __shfl_xor_sync(0xffffffffu, l[a], off);
#pragma unroll
    for (int c = 0; c < D / 64; ++c) {
      float y[4];
      tc::upk2(at.h ? o[H + a][c][0] : o[a][c][0], y[0], y[1]);
      tc::upk2(at.h ? o[H + a][c][1] : o[a][c][1], y[2], y[3]);
      const float4 z = *reinterpret_cast<const float4 *>(&sh.o[at.own<RPG>(a)][at.tx * 4 + 64 * c]);
      x[a][c][0] = y[0] + z.x;
      x[a][c][1] = y[1] + z.y;
      x[a][c][2] = y[2] + z.z;
      x[a][c][3] = y[3] + z.w;
    }
  }
}

}  // namespace simt
}  // namespace mgqa
