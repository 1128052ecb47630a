// Rows of a cache in 4 bits, and products with them on the tensor cores.
//
// A row of D features is a record of D/2 + 16 bytes: four groups of D/4 features,
// each with codes u in 0..15, a scale and a least value (fp16), x = scale u + least.
// The codes come first, two a byte (the even feature in the low half; D = 128: a
// group is 16 bytes; D = 64: 8 bytes, with those of groups 0 and 1, and of 2 and 3,
// by turns), then the four scales and the four least values.
//
// The raw bits of a code in the low bits of an fp16 are the number u 2^-24 (a
// subnormal), and one place higher u 2^-20, so four masks and a shift make eight
// codes exact tensor-core operands, with nothing subtracted and nothing rounded;
// the scales and least values come in beside the products:
//   s_j   = sum_g scale_jg <q_g, u_jg> + sum_g least_jg sum(q_g)
//   out_d = sum_j (p_j scale_jg(d)) u_jd + sum_j p_j least_jg(d)
// The least values' sums are products with the eight parameters of a record, taken
// as a row (or column) of 8. (As 16-bit rows, scaled and rounded, a value took 1.3
// instructions to unpack instead of 0.63, and lost 2^-9 of it.)
// A pitch of 80 (48) bytes spreads eight rows over all banks, so records are copied
// as they lie.
#pragma once

#include "common.cuh"

namespace mgqa {

template <int D>
struct Q4 {
  static constexpr int CODES = D / 2;        // bytes of codes
  static constexpr int REC = CODES + 16;     // bytes of a record
  static constexpr int CHUNKS = CODES / 16;  // 16-byte pieces of codes
  static constexpr int KS = D / 64;          // products of 16 features per group
  static constexpr int GW = D / 4;           // features of a group
  // Feature of value i of a query's fragment in group g: a lane (quad place tq) has
  // GW / 4 features of every group, one run of them.
  static MGQA_DEV int first(int g, int tq) { return g * GW + tq * (GW / 4); }
  // First feature of what a lane (gq) has of the outputs of chunk c, and how many
  // features follow it: half h adds the codes 2h and 2h + 1 of a 16-bit unit.
  static MGQA_DEV int out_feature(int c, int h, int gq) {
    return D == 128 ? 32 * c + 4 * gq + 2 * h : 16 * (2 * c + h) + 2 * gq;
  }
  static constexpr int group_of(int c, int h) { return D == 128 ? c : 2 * c + h; }
};

// Eight codes as four operand registers: the low and the next code of each 16-bit
// unit (worth 2^-24 and 2^-20), then those of its upper byte.
MGQA_DEV void q4_unpack(uint32_t w, uint32_t (&a)[4]) {
  a[0] = w & 0x000f000fu;
  a[1] = w & 0x00f000f0u;
  w >>= 8;
  a[2] = w & 0x000f000fu;
  a[3] = w & 0x00f000f0u;
}

// The same as (u - c) 2^-9, from[i]: -c 2^-9 (twice) of the codes of byte i of a unit; c a
// multiple of 1/64, so exact.
MGQA_DEV void q4_unpack_from(uint32_t w, const uint32_t (&from)[2], uint32_t (&a)[4]) {
  q4_unpack(w, a);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t up = i % 2 ? 0x68006800u : 0x78007800u;  // 2^11 or 2^15
    const __half2 x = __hfma2(*reinterpret_cast<const __half2 *>(&a[i]), *reinterpret_cast<const __half2 *>(&up),
                              *reinterpret_cast<const __half2 *>(&from[i / 2]));
    a[i] = *reinterpret_cast<const uint32_t *>(&x);
  }
}
// The same from the middle of all codes, (u - 8) 2^-9: normal numbers. (The tensor cores
// align a subnormal operand's products by the least exponent, which costs their sums some 8
// bits; fp32 calls: an error of 5.5e-6 of the outputs' size without.)
MGQA_DEV void q4_unpack_middle(uint32_t w, uint32_t (&a)[4]) {
  const uint32_t from[2] = {0xa400a400u, 0xa400a400u};
  q4_unpack_from(w, from, a);
}
template <bool MIDDLE>
MGQA_DEV void q4_codes(uint32_t w, uint32_t (&a)[4]) {
  if constexpr (MIDDLE) q4_unpack_middle(w, a);
  else q4_unpack(w, a);
}

// 2^k, k in [-126, 127].
MGQA_DEV float pow2i(int k) { return __int_as_float((k + 127) << 23); }

// One query row's operands in a lane (quad place tq): fp16 of q 2^k, the row's
// largest in [2^6, 2^7). A feature is off by at most 2^-27 of the row's largest: those of
// the second codes of a unit (see below) are divided by 16, and fp16's least step is 2^-24.
// (fp16 queries keep every bit down to 2^-16 of the largest, bf16 ones down to 2^-19.) fp32
// ones are two terms (22 bits, and 2^-31 of the largest), and meet codes from their
// middle, u - 8: the terms that cancel are small then (the tensor cores' sums truncate).
// Where codes count from 0 the second code of a unit is worth 16 times the first: its
// features are divided by that. `sums`: the groups' sums in two terms, for the least values
// (lanes tq 2 and 3), and 8 times that for the scales (0 where codes count from 0).
template <int D, bool SPLIT>
struct Q4Row {
  uint32_t a[4][Q4<D>::KS][2], b[SPLIT ? 4 : 1][Q4<D>::KS][2];  // b: second terms
  uint32_t sums[2];
  float down;  // 2^-k

  template <typename T>
  MGQA_DEV void load(const T *row, int tq, bool negate = false) {  // null: zeros. (The four lanes of a quad together.)
    constexpr int N = Q4<D>::GW / 4;  // features of a group
    float x[4][N];
    float top = 0.f;
#pragma unroll
    for (int g = 0; g < 4; ++g) {
      if (row) {
        const T *src = row + Q4<D>::first(g, tq);
        if constexpr (sizeof(T) == 4) {
#pragma unroll
          for (int i = 0; i < N; i += 4) {
            const float4 v = *reinterpret_cast<const float4 *>(src + i);
            x[g][i] = v.x; x[g][i + 1] = v.y; x[g][i + 2] = v.z; x[g][i + 3] = v.w;
          }
        } else if constexpr (N == 8) {
          unpack16_t<T>(*reinterpret_cast<const uint4 *>(src), x[g]);
        } else {
          const uint2 u = *reinterpret_cast<const uint2 *>(src);
          float f[8];
          unpack16_t<T>(make_uint4(u.x, u.y, 0u, 0u), f);
#pragma unroll
          for (int i = 0; i < 4; ++i) x[g][i] = f[i];
        }
      } else {
#pragma unroll
        for (int i = 0; i < N; ++i) x[g][i] = 0.f;
      }
#pragma unroll
      for (int i = 0; i < N; ++i) top = fmaxf(top, fabsf(x[g][i]));
    }
    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
    const int e = (int)(__float_as_uint(top) >> 23) - 127;  // (0: -127)
    const int k = min(6 - e, 120);
    const float up = negate ? -pow2i(k) : pow2i(k);
    down = pow2i(-k);
    float sum[4];
#pragma unroll
    for (int g = 0; g < 4; ++g) {
      sum[g] = 0.f;
#pragma unroll
      for (int i = 0; i < N; ++i) {
        x[g][i] *= up;
        sum[g] += x[g][i];
      }
      sum[g] += __shfl_xor_sync(0xffffffffu, sum[g], 1);
      sum[g] += __shfl_xor_sync(0xffffffffu, sum[g], 2);
#pragma unroll
      for (int s = 0; s < Q4<D>::KS; ++s)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          // D = 128: features {2s, 2s + 4}, {2s + 1, 2s + 5}; D = 64: {0, 2}, {1, 3}
          const float m = h && !SPLIT ? 0.0625f : 1.f;
          const float u = x[g][2 * s + h] * m, v = x[g][2 * s + h + (N == 8 ? 4 : 2)] * m;
          a[g][s][h] = pack2<__half>(u, v);
          if constexpr (SPLIT) {
            const float2 hi = __half22float2(*reinterpret_cast<const __half2 *>(&a[g][s][h]));
            b[g][s][h] = pack2<__half>(u - hi.x, v - hi.y);
          }
        }
    }
    sums[0] = sums[1] = 0u;
    if (SPLIT || tq >= 2) {
      const float by = tq < 2 ? 8.f : 1.f, u = by * (tq % 2 ? sum[2] : sum[0]), v = by * (tq % 2 ? sum[3] : sum[1]);
      sums[0] = pack2<__half>(u, v);
      const float2 hi = __half22float2(*reinterpret_cast<const __half2 *>(&sums[0]));
      sums[1] = pack2<__half>(u - hi.x, v - hi.y);
    }
  }
};

// Four halves at p (8-byte aligned, shared memory) as floats.
MGQA_DEV void q4_four(const unsigned char *p, float (&f)[4]) {
  const uint2 w = *reinterpret_cast<const uint2 *>(p);
  const float2 a = __half22float2(*reinterpret_cast<const __half2 *>(&w.x));
  const float2 b = __half22float2(*reinterpret_cast<const __half2 *>(&w.y));
  f[0] = a.x; f[1] = a.y; f[2] = b.x; f[3] = b.y;
}

// Scores of 16 keys with 8 query rows, unscaled (times the row's `down`): s[0], s[1]
// are key gq with rows 2 tq and 2 tq + 1, s[2], s[3] key gq + 8. least: the keys'
// parameters (word tq of each); u: their codes of chunk c, unpacked; sc: their scales.
// A piece at a time, so that unpacked codes serve several groups of rows.
template <int D, bool SPLIT>
struct Q4Scores {
  float s[4], acc[4];

  MGQA_DEV void least(const uint32_t (&p)[4], const uint32_t (&sums)[2]) {  // p: keys gq, gq + 8, and both again
    mma_16816_first<__half>(s, p[0], p[1], p[2], p[3], sums[0], sums[1]);
  }
  // q(g, i): both operand registers of product i of group g; q2: their second terms
  template <typename Q, typename Q2>
  MGQA_DEV void chunk(int c, const uint32_t (&u)[2][4], const float (&sc)[2][4], Q q, Q2 q2) {
    float part[4];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int g = Q4<D>::group_of(c, h), i = D == 128 ? h : 0;
      const uint2 b = q(g, i);
      if (D == 64 || h == 0) mma_16816_first<__half>(part, u[0][2 * h], u[1][2 * h], u[0][2 * h + 1], u[1][2 * h + 1], b.x, b.y);
      else mma_16816<__half>(part, u[0][2 * h], u[1][2 * h], u[0][2 * h + 1], u[1][2 * h + 1], b.x, b.y);
      if constexpr (SPLIT) {
        const uint2 b2 = q2(g, i);
        mma_16816<__half>(part, u[0][2 * h], u[1][2 * h], u[0][2 * h + 1], u[1][2 * h + 1], b2.x, b2.y);
      }
      if (D == 64 || h == 1) {  // the group is complete
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[e] = g == 0 ? part[e] * sc[e / 2][g] : fmaf(part[e], sc[e / 2][g], acc[e]);
      }
    }
  }
  MGQA_DEV void finish() {
#pragma unroll
    for (int e = 0; e < 4; ++e) s[e] = fmaf(acc[e], SPLIT ? 512.f : 16777216.f, s[e]);
  }
};

}  // namespace mgqa
