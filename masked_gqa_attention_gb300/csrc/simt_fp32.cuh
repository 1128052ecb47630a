// Register-tiled fp32 products of the CUDA-core attention kernels: 64 keys per
// tile, K and V in shared memory as TMA leaves them (boxes of 64 rows x 32
// floats, 128-byte swizzled), 256 threads. A thread (ty, tx) of the 16 x 16
// grid has query rows ty + 16 a and keys tx + 16 c.
// Every product is a packed pair of fp32 multiply-adds (one instruction for
// two), which leaves issue slots for the shared-memory reads: with single
// multiply-adds the loop was bound by issue at ~41 % of the fp32 rate.
#pragma once

#include "common.cuh"
#include "tc_ptx.cuh"

namespace mgqa {
namespace simt {

constexpr int kBox = 64 * 128;  // bytes of a box

MGQA_DEV void lds_pairs(uint64_t &a, uint64_t &b, const void *p) {  // 16 bytes as two pairs
  asm volatile("ld.shared.v2.u64 {%0, %1}, [%2];" : "=l"(a), "=l"(b) : "r"(smem_u32(p)));
}
MGQA_DEV float pair_sum(uint64_t x) {
  float a, b;
  tc::upk2(x, a, b);
  return a + b;
}

// s[a][c] = <q row ty + 16 a, key tx + 16 c>. QP: row pitch of q (floats).
template <int D, int RPT, int QP>
MGQA_DEV void scores(float (&s)[RPT][4], const float *q, const unsigned char *kt, int ty, int tx) {
  uint64_t acc[RPT][4];
#pragma unroll
  for (int a = 0; a < RPT; ++a)
#pragma unroll
    for (int c = 0; c < 4; ++c) acc[a][c] = 0ull;
  const unsigned char *krow = kt + tx * 128;
#pragma unroll
  for (int b = 0; b < D / 32; ++b)
#pragma unroll 4
    for (int d4 = 0; d4 < 8; ++d4) {
      uint64_t k0[4], k1[4];
      const int off = b * kBox + ((d4 ^ (tx & 7)) << 4);
#pragma unroll
      for (int c = 0; c < 4; ++c) lds_pairs(k0[c], k1[c], krow + off + c * (16 * 128));
#pragma unroll
      for (int a = 0; a < RPT; ++a) {
        uint64_t q0, q1;
        lds_pairs(q0, q1, q + (ty + 16 * a) * QP + b * 32 + d4 * 4);
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          acc[a][c] = tc::fma2(q0, k0[c], acc[a][c]);
          acc[a][c] = tc::fma2(q1, k1[c], acc[a][c]);
        }
      }
    }
#pragma unroll
  for (int a = 0; a < RPT; ++a)
#pragma unroll
    for (int c = 0; c < 4; ++c) s[a][c] = pair_sum(acc[a][c]);
}

// o[a][c] (features 4 tx + 64 c .. + 3 as two pairs) += the weights of row
// ty + 16 a times V. w: weights [row][key], each twice in a row (pitch WP
// floats). ok: which keys count (the rows of the others may hold anything).
template <int D, int RPT, int WP>
MGQA_DEV void values(uint64_t (&o)[RPT][D / 64][2], const float *w, const unsigned char *vt, int ty, int tx,
                     uint32_t ok_lo, uint32_t ok_hi) {
  const bool clean = (ok_lo & ok_hi) == 0xffffffffu;
#pragma unroll 4
  for (int k = 0; k < 64; k += 2) {
    uint64_t v[2][D / 64][2];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const unsigned char *vr = vt + (tx >> 3) * kBox + (k + e) * 128 + (((tx & 7) ^ ((k + e) & 7)) << 4);
#pragma unroll
      for (int c = 0; c < D / 64; ++c) lds_pairs(v[e][c][0], v[e][c][1], vr + c * 2 * kBox);
      if (!clean && !(((k < 32 ? ok_lo : ok_hi) >> ((k + e) & 31)) & 1u))
#pragma unroll
        for (int c = 0; c < D / 64; ++c) v[e][c][0] = v[e][c][1] = 0ull;
    }
#pragma unroll
    for (int a = 0; a < RPT; ++a) {
      uint64_t w0, w1;
      lds_pairs(w0, w1, w + (ty + 16 * a) * WP + 2 * k);
#pragma unroll
      for (int c = 0; c < D / 64; ++c) {
        o[a][c][0] = tc::fma2(w0, v[0][c][0], o[a][c][0]);
        o[a][c][1] = tc::fma2(w0, v[0][c][1], o[a][c][1]);
        o[a][c][0] = tc::fma2(w1, v[1][c][0], o[a][c][0]);
        o[a][c][1] = tc::fma2(w1, v[1][c][1], o[a][c][1]);
      }
    }
  }
}

MGQA_DEV uint64_t mul2(uint64_t a, float f) {
  uint64_t d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(tc::pk2(f, f)));
  return d;
}

// One row of the running softmax over a tile's scores, held by the 16 threads
// of a half-warp (4 keys each, in log2 units, masked ones -inf): the weights go
// to w (twice each), the factor for what was summed before is returned.
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
    *reinterpret_cast<float2 *>(w + 2 * (tx + 16 * c)) = make_float2(x, x);
  }
  return f;
}

}  // namespace simt
}  // namespace mgqa
