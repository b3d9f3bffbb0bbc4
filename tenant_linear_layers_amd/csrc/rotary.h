// The rotation of pairs of dims by the angle of a token's position:
//   (a, b) -> (a cos - b sin, b cos + a sin)
// The two products of a member are rounded apart (no fused multiply-add): the
// bits are then the same whichever kernel turns a row, and those of the same
// products and sums taken one by one.
#pragma once

#include "common.h"
#include "layer.h"

namespace bd {

typedef f32x4 f32x4_any __attribute__((aligned(4)));

__device__ __forceinline__ float turned_first(float a, float b, float c, float s) {
#pragma clang fp contract(off)
  return a * c - b * s;
}
__device__ __forceinline__ float turned_second(float a, float b, float c, float s) {
#pragma clang fp contract(off)
  return b * c + a * s;
}

// N cosines and sines from a table's place; NaN for no place.
template <int N>
struct Angles {
  float c[N], s[N];
  __device__ __forceinline__ void load(const float* t, int n) {
#pragma unroll
    for (int i = 0; i < N; ++i) c[i] = s[i] = NAN;
    if (!t) return;
    if (n >= N) {
#pragma unroll
      for (int i = 0; i < N; i += 2) {
        const f32x4 v = *reinterpret_cast<const f32x4_any*>(t + 2 * i);
        c[i] = v[0];
        s[i] = v[1];
        c[i + 1] = v[2];
        s[i + 1] = v[3];
      }
    } else {
#pragma unroll
      for (int i = 0; i < N; ++i)
        if (i < n) {
          c[i] = t[2 * i];
          s[i] = t[2 * i + 1];
        }
    }
  }
};

// A table's row for a position, or nullptr outside of it.
__device__ __forceinline__ const float* table_row(const float* table, int length, int rot, int pos) {
  return pos >= 0 && pos < length ? table + (int64_t)pos * rot : nullptr;
}

// Up to eight elements from p, and to it.
__device__ __forceinline__ u32x4 ld_upto8(const uint16_t* p, int n) {
  if (n >= 8) return *reinterpret_cast<const u32x4_any*>(p);
  u32x4 v = {0u, 0u, 0u, 0u};
#pragma unroll
  for (int e = 0; e < 8; ++e)
    if (e < n) v[e >> 1] |= (uint32_t)p[e] << ((e & 1) << 4);
  return v;
}
__device__ __forceinline__ void st_upto8(uint16_t* p, u32x4 v, int n) {
  if (n >= 8) {
    *reinterpret_cast<u32x4_any*>(p) = v;
    return;
  }
#pragma unroll
  for (int e = 0; e < 8; ++e)
    if (e < n) p[e] = (uint16_t)(v[e >> 1] >> ((e & 1) << 4));
}

// Thread i of a call's rotation.  A unit is eight pairs of a row (16 values
// interleaved, two runs of eight otherwise), or 16 dims behind the pairs that
// are copied; a thread takes one unit of every parts-th head, whose cosines
// and sines it reads once.  Each value is read and written by one thread, which
// reads a batch of heads before it writes them: out may be x.
template <bool INTERLEAVED>
__device__ __forceinline__ void rotate_unit(const RotaryArgs& a, int i) {
  constexpr int HEADS = 4;
  const int rest = a.by_units.of(i), u = i - rest * a.units;
  const int64_t token = a.by_parts.of(rest);
  const int part = rest - (int)token * a.parts;
  if (token >= a.tokens) return;
  const bool turns = u < a.turning;
  const int half = a.rot >> 1;
  const int first = turns ? (INTERLEAVED ? 16 * u : 8 * u) : a.rot + 16 * (u - a.turning);
  const int second = turns && !INTERLEAVED ? first + half : first + 8;
  const int left = turns ? half - 8 * u : a.dim - first;   // pairs, or dims
  const int n0 = turns && INTERLEAVED ? 2 * left : left;
  const int n1 = turns && !INTERLEAVED ? left : n0 - 8;
  Angles<8> t;
  if (turns) {
    const float* row = table_row(a.table, a.length, a.rot, a.positions[token]);
    t.load(row ? row + 16 * u : nullptr, left);
  }
  const uint16_t* x = a.x + token * a.x_token_stride;
  uint16_t* o = a.out + token * a.out_token_stride;
  for (int h0 = part; h0 < a.heads; h0 += HEADS * a.parts) {
    u32x4 v[HEADS][2];
#pragma unroll
    for (int k = 0; k < HEADS; ++k) {
      const int64_t h = h0 + k * a.parts;
      if (h < a.heads) {
        v[k][0] = ld_upto8(x + h * a.x_head_stride + first, n0);
        v[k][1] = ld_upto8(x + h * a.x_head_stride + second, n1);
      }
    }
#pragma unroll
    for (int k = 0; k < HEADS; ++k) {
      const int64_t h = h0 + k * a.parts;
      if (h >= a.heads) break;
      if (turns) {
        float f[16];   // the unit's values in the order of v
#pragma unroll
        for (int d = 0; d < 8; ++d) {
          f[2 * d] = lo16(v[k][d >> 2][d & 3]);
          f[2 * d + 1] = hi16(v[k][d >> 2][d & 3]);
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const int p = INTERLEAVED ? 2 * e : e, q = INTERLEAVED ? 2 * e + 1 : e + 8;
          const float fa = f[p], fb = f[q];
          f[p] = turned_first(fa, fb, t.c[e], t.s[e]);
          f[q] = turned_second(fa, fb, t.c[e], t.s[e]);
        }
#pragma unroll
        for (int d = 0; d < 8; ++d) v[k][d >> 2][d & 3] = cvt_pk_bf16(f[2 * d], f[2 * d + 1]);
      }
      st_upto8(o + h * a.out_head_stride + first, v[k][0], n0);
      st_upto8(o + h * a.out_head_stride + second, v[k][1], n1);
    }
  }
}

// Fills in what a launch's threads go by; their number for `tokens` of them.
// Rows are shared by the threads of a token only as far as that leaves the
// card full: the angles, 64 bytes a unit of 32, are then read for fewer rows.
inline int64_t rotary_plan(RotaryArgs& a) {
  a.turning = (a.rot / 2 + 7) / 8;
  a.units = a.turning + (a.x == a.out ? 0 : (a.dim - a.rot + 15) / 16);
  int each = 1;
  while (each < 8 && a.tokens * a.units * a.heads / (2 * each) >= (int64_t(1) << 18)) each *= 2;
  a.parts = (a.heads + each - 1) / each;
  a.by_units = divisor(a.units);
  a.by_parts = divisor(a.parts);
  return (int64_t)a.units * a.parts;
}

}  // namespace bd
