// The paged key/value cache: rows [dim] of one head and token, in bf16, in
// e4m3 with one power-of-two scale per row, or in e2m1 with one per 32 dims.
//
// The kernels move each row once and are bound by HBM (2 bytes a value on the
// bf16 side, 2, 1 + 1/dim or 1/2 + 1/32 on the cache's) or, for a batch of
// single tokens, by the launch.  dim / 8 neighbouring lanes hold a row of k and
// of v: one 16-byte access a lane and row on the bf16 side, and a group's largest
// magnitude by lane exchanges, so a row needs no LDS.  Neighbouring rows of a
// token are its heads, contiguous on the side of the tokens.  8 heads of 128: 64
// tokens into 8 or 4 bits take 3.2 and 3.0 us, 2048 4.4 and 4.1, 16001 19.6 and 18.8, back
// 17.3 and 19.0 (4 bits, from cold memory and single slots: 22.8 and 20.7, 3.6 and
// 4.0 TB/s of what is needed; a slot's 4 bytes of scales move 32 and its 64 of
// codes half a line).
#include "common.h"
#include "e2m1.h"
#include "e4m3.h"
#include "layer.h"
#include "rotary.h"

namespace bd {
namespace {

// Thread i's place: token, head and eight values, of k and of v (one row's place
// for both, and two loads on their way).
struct Place {
  int head, piece;
  int64_t token, row;  // row of the caches, or -1 for a slot outside them
};

template <int D>
__device__ __forceinline__ bool place(const KvArgs& a, int i, Place& p) {
  constexpr int L = D / 8;
  const int token = a.by_token.of(i);
  const int j = i - token * a.by_token.by;
  p.token = token;
  p.piece = j % L;
  p.head = j / L;
  return token < a.tokens;
}

// The place's row of the caches.  Writes look it up before they read a token, so one
// that is passed over costs its slot's four bytes: of 16001 tokens, half of them
// padding, a write takes 12 us, with the rows read beside the slots 16 to 17, and an
// append (64 heads and 8) 115 to 119 for 121 to 125.  Without padding that is up to
// 0.1 us of 3 for few tokens, and nothing or up to 1% for many.
__device__ __forceinline__ void find_row(const KvArgs& a, Place& p) {
  const int slot = a.slots[p.token];
  const int page = a.by_page.of(max(slot, 0));
  p.row = slot < 0 || slot >= a.n_slots
              ? -1
              : ((int64_t)page * a.heads + p.head) * a.page + (slot - page * a.page);
}

// The larger of a lane's value and its neighbour's, one or two lanes on in its
// four.
template <int STEP>
__device__ __forceinline__ uint32_t quad_max(uint32_t v) {
  constexpr int kOther = STEP == 1 ? 0xB1 : 0x4E;   // lanes 1 0 3 2, lanes 2 3 0 1
  return max(v, (uint32_t)__builtin_amdgcn_mov_dpp((int)v, kOther, 0xF, 0xF, true));
}

__device__ __forceinline__ const uint16_t* source(const KvArgs& a, const Place& p, int w) {
  return a.src[w] + p.token * a.token_stride[w] + p.head * a.head_stride[w];
}

__device__ __forceinline__ void to_floats(u32x4 v, float (&f)[8]) {
#pragma unroll
  for (int d = 0; d < 4; ++d) {
    f[2 * d] = lo16(v[d]);
    f[2 * d + 1] = hi16(v[d]);
  }
}

// Eight values of a row into cache w in 8 or 4 bits.
template <int D, int BITS>
__device__ __forceinline__ void put(const KvArgs& a, const Place& p, int w, float (&f)[8]) {
  if constexpr (BITS == 8) {
    float m = 0.f;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      f[e] = hold_e4m3(f[e]);
      m = fmaxf(m, fabsf(f[e]));
    }
#pragma unroll
    for (int o = 1; o < D / 8; o <<= 1) m = fmaxf(m, __shfl_xor(m, o));
    const uint32_t sb = scale_byte(m);
    const float is = inv_scale(sb);
    const u32x2 o = {pack_e4m3(f[0] * is, f[1] * is, f[2] * is, f[3] * is),
                     pack_e4m3(f[4] * is, f[5] * is, f[6] * is, f[7] * is)};
    *reinterpret_cast<u32x2*>(static_cast<uint8_t*>(a.cache[w]) + p.row * D + p.piece * 8) = o;
    if (p.piece == 0) a.scale[w][p.row] = (uint8_t)sb;
  } else {
    uint32_t m = 0u;   // a magnitude's bits order as it does, a NaN's last
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      f[e] = hold_e2m1(f[e]);
      m = max(m, __float_as_uint(f[e]) & 0x7FFFFFFFu);
    }
    m = quad_max<2>(quad_max<1>(m));   // four lanes hold a group
    const uint32_t sb = scale_byte4(m);
    *reinterpret_cast<uint32_t*>(static_cast<uint8_t*>(a.cache[w]) + p.row * (D / 2) +
                                 p.piece * 4) =
        sb == kNanScale ? 0u : pack_e2m1(f, __uint_as_float(sb << 23));
    if (p.piece % (kGroup4 / 8) == 0)
      a.scale[w][p.row * (D / kGroup4) + p.piece / (kGroup4 / 8)] = (uint8_t)sb;
  }
}

template <int D>
__device__ __forceinline__ void put16(const KvArgs& a, const Place& p, int w, u32x4 v) {
  *reinterpret_cast<u32x4*>(static_cast<uint16_t*>(a.cache[w]) + p.row * D + p.piece * 8) = v;
}

template <int D, int BITS>
__global__ __launch_bounds__(256) void kv_write_kernel(const KvArgs a) {
  Place p;
  if (!place<D>(a, (int)(blockIdx.x * 256 + threadIdx.x), p)) return;
  find_row(a, p);
  if (p.row < 0) return;   // whole rows leave together
  u32x4 v[2];
#pragma unroll
  for (int w = 0; w < 2; ++w)
    v[w] = *reinterpret_cast<const u32x4_any*>(source(a, p, w) + p.piece * 8);
#pragma unroll
  for (int w = 0; w < 2; ++w) {
    if constexpr (BITS == 16) {
      put16<D>(a, p, w, v[w]);
    } else {
      float f[8];
      to_floats(v[w], f);
      put<D, BITS>(a, p, w, f);
    }
  }
}

template <int D, int BITS>
__global__ __launch_bounds__(256) void kv_read_kernel(const KvArgs a) {
  Place p;
  if (!place<D>(a, (int)(blockIdx.x * 256 + threadIdx.x), p)) return;
  find_row(a, p);
  u32x4 v[2];
#pragma unroll
  for (int w = 0; w < 2; ++w) v[w] = u32x4{0x7FC07FC0u, 0x7FC07FC0u, 0x7FC07FC0u, 0x7FC07FC0u};
  if (p.row >= 0) {   // else there is no such slot: NaN
#pragma unroll
    for (int w = 0; w < 2; ++w) {
      const uint8_t* rows = static_cast<const uint8_t*>(a.cache[w]);
      if constexpr (BITS == 8) {
        const u32x2 c = *reinterpret_cast<const u32x2*>(rows + p.row * D + p.piece * 8);
        const float s = __uint_as_float((uint32_t)a.scale[w][p.row] << 23);
        v[w] = u32x4{bf16x2_of_e4m3<false>(c[0], s), bf16x2_of_e4m3<true>(c[0], s),
                     bf16x2_of_e4m3<false>(c[1], s), bf16x2_of_e4m3<true>(c[1], s)};
      } else if constexpr (BITS == 4) {
        const uint32_t c =
            *reinterpret_cast<const uint32_t*>(rows + p.row * (D / 2) + p.piece * 4);
        const uint32_t sb = a.scale[w][p.row * (D / kGroup4) + p.piece / (kGroup4 / 8)];
        v[w] = bf16x8_of_e2m1(c, __uint_as_float(sb << 23));
      } else {
        v[w] = *reinterpret_cast<const u32x4*>(rows + (p.row * D + p.piece * 8) * 2);
      }
    }
  }
#pragma unroll
  for (int w = 0; w < 2; ++w)
    *reinterpret_cast<u32x4*>(a.dst[w] + (p.token * a.heads + p.head) * D + p.piece * 8) = v[w];
}

// Eight values of a row of k, turned by its token's angles.
template <int D, bool INTERLEAVED>
__device__ __forceinline__ void turn(const RotaryArgs& r, int64_t token, const uint16_t* row,
                                     int d0, float (&f)[8]) {
  if (d0 >= r.rot) return;
  const float* t = table_row(r.table, r.length, r.rot, r.positions[token]);
  const int half = r.rot >> 1;
  if constexpr (INTERLEAVED) {
    const int n = min((r.rot - d0) >> 1, 4);
    Angles<4> g;
    g.load(t ? t + d0 : nullptr, n);
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (e < n) {
        const float a = f[2 * e], b = f[2 * e + 1];
        f[2 * e] = turned_first(a, b, g.c[e], g.s[e]);
        f[2 * e + 1] = turned_second(a, b, g.c[e], g.s[e]);
      }
  } else if (half % 8 == 0) {   // the eight are all first or all second members
    const bool second = d0 >= half;
    const int pair = second ? d0 - half : d0;
    float o[8];
    to_floats(*reinterpret_cast<const u32x4_any*>(row + (second ? pair : pair + half)), o);
    Angles<8> g;
    g.load(t ? t + 2 * pair : nullptr, 8);
#pragma unroll
    for (int e = 0; e < 8; ++e)
      f[e] = second ? turned_second(o[e], f[e], g.c[e], g.s[e])
                    : turned_first(f[e], o[e], g.c[e], g.s[e]);
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int d = d0 + e;
      if (d < r.rot) {
        const bool second = d >= half;
        const int pair = second ? d - half : d;
        const float o = __uint_as_float((uint32_t)row[second ? pair : pair + half] << 16);
        const float c = t ? t[2 * pair] : NAN, s = t ? t[2 * pair + 1] : NAN;
        f[e] = second ? turned_second(o, f[e], c, s) : turned_first(f[e], o, c, s);
      }
    }
  }
}

// The first q_groups workgroups turn the queries, the others put rows into the
// cache: one launch for what a step has between its QKV product and its
// attention.  The queries, most of the bytes, go first: 2048 tokens of 64 heads
// 16.2 us, the other way round 18.1 (16001 tokens 156 and 151).
template <int D, int BITS, bool INTERLEAVED>
__global__ __launch_bounds__(256) void kv_append_kernel(const KvArgs a, const RotaryArgs r,
                                                        const unsigned q_groups) {
  if (blockIdx.x < q_groups) {
    rotate_unit<INTERLEAVED>(r, (int)(blockIdx.x * 256 + threadIdx.x));
    return;
  }
  Place p;
  if (!place<D>(a, (int)((blockIdx.x - q_groups) * 256 + threadIdx.x), p)) return;
  find_row(a, p);
  if (p.row < 0) return;   // whole rows leave together
  const uint16_t *k = source(a, p, 0), *v = source(a, p, 1);
  float f[2][8];
  to_floats(*reinterpret_cast<const u32x4_any*>(k + p.piece * 8), f[0]);
  to_floats(*reinterpret_cast<const u32x4_any*>(v + p.piece * 8), f[1]);
  turn<D, INTERLEAVED>(r, p.token, k, p.piece * 8, f[0]);
#pragma unroll
  for (int w = 0; w < 2; ++w) {
    if constexpr (BITS == 16) {
      u32x4 o;
#pragma unroll
      for (int d = 0; d < 4; ++d) o[d] = cvt_pk_bf16(f[w][2 * d], f[w][2 * d + 1]);
      put16<D>(a, p, w, o);
    } else {
      put<D, BITS>(a, p, w, f[w]);
    }
  }
}

// A thread's index is an int: more tokens than that go in several launches, of
// 2^30 threads at most.
template <int D, int BITS, bool WRITE>
hipError_t run(const KvArgs& a, hipStream_t s) {
  const int64_t per = (int64_t)a.heads * (D / 8);   // threads of a token
  const int64_t most = (int64_t(1) << 30) / per;
  for (int64_t at = 0; at < a.tokens; at += most) {
    KvArgs b = a;
    b.by_token = divisor((int)per);
    b.by_page = divisor(a.page);
    b.tokens = a.tokens - at < most ? a.tokens - at : most;
    b.slots += at;
    for (int w = 0; w < 2; ++w) {
      if (WRITE) b.src[w] += at * a.token_stride[w];
      else b.dst[w] += at * a.heads * D;
    }
    const unsigned grid = (unsigned)((b.tokens * per + 255) / 256);
    if (WRITE) kv_write_kernel<D, BITS><<<grid, 256, 0, s>>>(b);
    else kv_read_kernel<D, BITS><<<grid, 256, 0, s>>>(b);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

template <int D, int BITS>
hipError_t run_append(const KvArgs& a, RotaryArgs r, hipStream_t s) {
  const int64_t per = (int64_t)a.heads * (D / 8), per_q = rotary_plan(r);
  const int64_t most = (int64_t(1) << 30) / (per > per_q ? per : per_q);
  for (int64_t at = 0; at < a.tokens; at += most) {
    KvArgs b = a;
    RotaryArgs q = r;
    b.by_token = divisor((int)per);
    b.by_page = divisor(a.page);
    b.tokens = q.tokens = a.tokens - at < most ? a.tokens - at : most;
    b.slots += at;
    q.positions += at;
    for (int w = 0; w < 2; ++w) b.src[w] += at * a.token_stride[w];
    q.x += at * r.x_token_stride;
    q.out += at * r.out_token_stride;
    const unsigned turns = (unsigned)((b.tokens * per_q + 255) / 256);
    const unsigned grid = turns + (unsigned)((b.tokens * per + 255) / 256);
    if (r.interleaved) kv_append_kernel<D, BITS, true><<<grid, 256, 0, s>>>(b, q, turns);
    else kv_append_kernel<D, BITS, false><<<grid, 256, 0, s>>>(b, q, turns);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

template <int D, bool WRITE>
hipError_t pick(const KvArgs& a, hipStream_t s) {
  return a.bits == 16  ? run<D, 16, WRITE>(a, s)
         : a.bits == 8 ? run<D, 8, WRITE>(a, s)
                       : run<D, 4, WRITE>(a, s);
}

template <int D>
hipError_t pick_append(const KvArgs& a, const RotaryArgs& q, hipStream_t s) {
  return a.bits == 16  ? run_append<D, 16>(a, q, s)
         : a.bits == 8 ? run_append<D, 8>(a, q, s)
                       : run_append<D, 4>(a, q, s);
}

}  // namespace

hipError_t launch_kv_write(const KvArgs& a, hipStream_t s) {
  return a.dim == 64 ? pick<64, true>(a, s) : pick<128, true>(a, s);
}
hipError_t launch_kv_read(const KvArgs& a, hipStream_t s) {
  return a.dim == 64 ? pick<64, false>(a, s) : pick<128, false>(a, s);
}
hipError_t launch_kv_append(const KvArgs& a, const RotaryArgs& q, hipStream_t s) {
  return a.dim == 64 ? pick_append<64>(a, q, s) : pick_append<128>(a, q, s);
}

}  // namespace bd
