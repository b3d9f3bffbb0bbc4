// Attention of new tokens over the paged key/value cache in bf16 or e4m3; the
// definition, the plan and the layout of the products are in attention_plan.h.
#include <type_traits>

#include "attention_plan.h"
#include "common.h"
#include "e4m3.h"
#include "layer.h"

namespace bd {
namespace {

// ------------------------------------------------------------------ few rows
// Tiles of 16 rows.  The NW waves of a workgroup take 32-key steps of the
// piece in turn, each through its own ring of U stages in LDS: rows go there
// straight from HBM (16 bytes a lane, whole rows in order, so a load is
// coalesced; only the pieces of a row are permuted) and are read back as
// matrix operands, so there is no barrier until the waves' sums are joined.
//
// Bound by HBM: 64 sequences in 8 bits (688 MB) take 137 us, 5.0 TB/s, 32 in
// bf16 (795 MB) 142 us, 5.6 TB/s (a copy reaches 4.9 on this card); the CUs
// stand idle a fifth of the time at the ends.  A single token at 4097 keys,
// 10.1 us, is a chain of latencies: plan, page table, K, V, joins.
template <int D, bool Q8, int NW, int U>
__global__ __launch_bounds__(NW * 64) void attend_rows16_kernel(const AttnArgs a, const Cut c) {
  constexpr int R = 16;
  constexpr int ROWB = Q8 ? D : 2 * D;
  constexpr int P = ROWB / 16;              // 16-byte pieces of a row
  constexpr int KPI = 64 / P;               // keys per staging instruction
  constexpr int IPH = 16 / KPI;             // staging instructions per 16 keys
  constexpr int HALF = 2 * IPH + (Q8 ? 2 : 0);   // loads of K, and of V, per step
  constexpr int STAGE = 32 * ROWB;          // one of K, V
  constexpr int RED = NW * R * (D + 2) * 4;
  constexpr int SMEM = NW * U * 2 * STAGE > RED ? NW * U * 2 * STAGE : RED;
  __shared__ __attribute__((aligned(16))) char smem[SMEM];

  Item it;
  if (!find_item<false>(a, c, a.first + (int)blockIdx.x, it)) return;
  const int lane = threadIdx.x & 63;
  const int wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int n = lane & 15, g4 = lane >> 4;
  const Tile t = tile_of(a, it.q0, it.n, it.len, it.tile, R);
  int lo, hi, kbeg, steps, vis_hi;   // of a pass

  // Q^T: lane n's row, the dims that the lane's K pieces hold.
  u32x4 qf[D / 32];
  const int my = min(n, t.rows - 1);
  const int qi = a.by_group.of(t.row0 + my);
  const uint16_t* qp =
      a.q + (int64_t)(t.first_q + qi) * a.q_token_stride +
      (int64_t)(it.head * a.group + (t.row0 + my) - qi * a.group) * a.q_head_stride;
#pragma unroll
  for (int s = 0; s < D / 32; ++s) {
    const int d0 = Q8 ? 64 * (s >> 1) + 16 * g4 + 8 * (s & 1) : 32 * s + 8 * g4;
    qf[s] = *reinterpret_cast<const u32x4_any*>(qp + d0);
  }
  const int pos = t.pos0 + qi;
  const int vis_lo = a.window ? pos - a.window + 1 : 0;

  char* ring = smem + wv * U * 2 * STAGE;
  int voff[IPH];
#pragma unroll
  for (int j = 0; j < IPH; ++j) {
    const int key = j * KPI + lane / P;
    voff[j] = key * ROWB + (((lane % P) ^ swizzle<ROWB>(key)) << 4);
  }
  uint32_t ks[U][2], vs[U][2];
  bool bad = false;
  int blocks = -1;   // lane 2 i + h: rows / 16 of the cache for half h of step i (mod 32)

  auto issue = [&](int i, int u, bool first) {
    if ((i & 31) == 0) {
      const int64_t key = (int64_t)kbeg + (int64_t)32 * NW * (i + (lane >> 1)) + 16 * (lane & 1);
      blocks = -1;
      if (key < hi) {
        const int at = a.by_page.of((int)key);
        const int page = a.table[(int64_t)it.b * a.width + at];
        if (page >= 0 && page < a.pages)
          blocks = (int)((((int64_t)page * a.kv_heads + it.head) * a.page + (key - at * a.page)) >>
                         4);
        else  // a page that the cache lacks: the rows that see it are NaN
          bad |= key + 16 > lo;
      }
    }
    const int key0 = kbeg + 32 * NW * i;
    char* st = ring + u * 2 * STAGE;
    int blk[2], keys[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      blk[h] = __builtin_amdgcn_readlane(blocks, 2 * (i & 31) + h);
      keys[h] = __builtin_amdgcn_readfirstlane(
          blk[h] < 0 || i >= steps ? 0 : min(max(hi - key0 - 16 * h, 0), 16));
      blk[h] = max(blk[h], 0);
    }
#pragma unroll
    for (int w = 0; w < 2; ++w) {
      if (Q8) {
#pragma unroll
        for (int h = 0; h < 2; ++h)
          (w ? vs : ks)[u][h] =
              bload32(a.scale[w] + (int64_t)blk[h] * 16, (keys[h] + 3) & ~3, 4 * g4, 0);
      }
#pragma unroll
      for (int h = 0; h < 2; ++h) {
#pragma unroll
        for (int j = 0; j < IPH; ++j) {
          // keys below lo read as zero (their rows may be anything), like
          // those from hi on, which lie past the resource
          const bool below = first && key0 + 16 * h + j * KPI + lane / P < lo;
          lds_bload16(a.cache[w] + (int64_t)blk[h] * (16 * ROWB), keys[h] * ROWB,
                      below ? 1 << 30 : voff[j], 0, st + w * STAGE + (h * IPH + j) * 1024);
        }
      }
      // the waits below count on K's loads before V's
      __builtin_amdgcn_sched_barrier(0);
    }
  };

  f32x4 acc[D / 16];
  float m, l;

  auto step = [&](int i, int u) {
    const int key0 = kbeg + 32 * NW * i;
    const char* kst = ring + u * 2 * STAGE;
    char* vst = ring + u * 2 * STAGE + STAGE;
    float s[8];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      f32x4 z = {0.f, 0.f, 0.f, 0.f};
      const int key = 16 * h + n;
#pragma unroll
      for (int p = 0; p < P / 4; ++p) {
        const u32x4 k4 = *reinterpret_cast<const u32x4*>(
            kst + key * ROWB + (((4 * p + g4) ^ swizzle<ROWB>(key)) << 4));
        if (Q8) {
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const u32x4 kf = {bf16x2_of_e4m3<false>(k4[2 * e], 1.f),
                              bf16x2_of_e4m3<true>(k4[2 * e], 1.f),
                              bf16x2_of_e4m3<false>(k4[2 * e + 1], 1.f),
                              bf16x2_of_e4m3<true>(k4[2 * e + 1], 1.f)};
            z = mfma16(kf, qf[2 * p + e], z);
          }
        } else {
          z = mfma16(k4, qf[p], z);
        }
      }
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        float v = z[r] * a.scale_log2;
        if (Q8) v *= scale_of(ks[u][h], r);
        s[4 * h + r] = v;
      }
    }
    // a mask only where some row of the tile sees part of the step
    if (key0 + 32 > t.all_hi || key0 < t.all_lo || key0 + 32 > hi) {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int j = key0 + 16 * (e >> 2) + 4 * g4 + (e & 3);
        s[e] = j < vis_hi && j >= vis_lo ? s[e] : -INFINITY;
      }
    }
    float top = s[0];
#pragma unroll
    for (int e = 1; e < 8; ++e) top = fmaxf(top, s[e]);
    // The reference moves only when a score passes it by 2^6 or more: until
    // then the weights stay below 2^6, far from the limits of float32 and
    // bf16, and no lane exchange or rescaling is needed.
    if (__ballot(top > m + 6.f)) {
      top = fmaxf(top, __shfl_xor(top, 16));
      top = fmaxf(top, __shfl_xor(top, 32));
      const float m1 = fmaxf(m, top);
      const float f = m1 == -INFINITY ? 1.f : __builtin_amdgcn_exp2f(m - m1);
      m = m1;
      l *= f;
#pragma unroll
      for (int d = 0; d < D / 16; ++d) acc[d] *= f;
    }
    const float ref = m == -INFINITY ? 0.f : m;
    u32x4 pf;
#pragma unroll
    for (int e = 0; e < 8; e += 2) {
      s[e] = __builtin_amdgcn_exp2f(s[e] - ref);
      s[e + 1] = __builtin_amdgcn_exp2f(s[e + 1] - ref);
      pf[e >> 1] = weights(s[e], s[e + 1], l);
      if (Q8) {
        // a weight of 0 stays 0 whatever the scale of a row that is not there;
        // times a power of two the rounded weights are the rounded products
#pragma unroll
        for (int f = e; f < e + 2; ++f)
          s[f] = s[f] > 0.f ? s[f] * scale_of(vs[u][f >> 2], f & 3) : 0.f;
        pf[e >> 1] = cvt_pk_bf16(s[e], s[e + 1]);
      }
    }
    wait_loads<HALF * 2 * (U - 1)>();
#pragma unroll
    for (int d4 = 0; d4 < D / 16; d4 += 4) {   // four tiles of 16 dims
      u32x4 vf[4];
      uint32_t at[4];
      if (Q8) {
        // eight keys (4 g4 + 0..3 of both halves) of one dim per lane
        const int key = 16 * (n >> 3) + 4 * g4 + ((n >> 1) & 3);
#pragma unroll
        for (int e = 0; e < 4; ++e)
          at[e] = lds_address(vst + key * ROWB + (((d4 + e) ^ swizzle<ROWB>(key)) << 4) +
                              8 * (n & 1));
        u32x2 v2[4];
        read_tr8(at, v2);
#pragma unroll
        for (int e = 0; e < 4; ++e)
          vf[e] = u32x4{bf16x2_of_e4m3<false>(v2[e][0], 1.f), bf16x2_of_e4m3<true>(v2[e][0], 1.f),
                        bf16x2_of_e4m3<false>(v2[e][1], 1.f), bf16x2_of_e4m3<true>(v2[e][1], 1.f)};
      } else {
        const int key = 4 * g4 + (n >> 2);
#pragma unroll
        for (int e = 0; e < 4; ++e)
          at[e] = lds_address(
              vst + key * ROWB +
              (((2 * (d4 + e) + ((n >> 1) & 1)) ^ swizzle<ROWB>(key)) << 4) + 8 * (n & 1));
        read_tr16<16 * ROWB>(at, vf);
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[d4 + e] = mfma16(vf[e], pf, acc[d4 + e]);
    }
  };

  int only = -1;   // the query of this pass, or all
  for (;;) {
    piece_range(t, it.piece, it.pieces, lo, hi);
    if (only >= 0) query_range(a, t, only, lo, hi);
    lo = __builtin_amdgcn_readfirstlane(lo);
    hi = __builtin_amdgcn_readfirstlane(hi);
    kbeg = (lo & ~31) + 32 * wv;
    steps = hi > kbeg ? (hi - kbeg + 32 * NW - 1) / (32 * NW) : 0;
    vis_hi = min(pos + 1, hi);
#pragma unroll
    for (int d = 0; d < D / 16; ++d) acc[d] = f32x4{0.f, 0.f, 0.f, 0.f};
    m = -INFINITY;
    l = 0.f;
    if (steps > 0) {
#pragma unroll
      for (int u = 0; u < U - 1; ++u) issue(u, u, u == 0);
      for (int i0 = 0; i0 < steps; i0 += U) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const int i = i0 + u;
          // the stage to be filled was read by the step before: those reads are
          // complete before loads may write it (a load to LDS is not ordered
          // after earlier reads of its wave)
          wait_lds();
          // past the last step the loads have no rows left and read nothing:
          // every step issues the same number
          issue(i + U - 1, (u + U - 1) % U, false);
          if (i < steps) {
            wait_loads<HALF * 2 * (U - 1) + HALF>();
            step(i, u);
          }
        }
      }
    }
    wait_loads<0>();
    if (__ballot(bad)) l = NAN;
    l += __shfl_xor(l, 16);
    l += __shfl_xor(l, 32);
    if (only < 0 && (t.all_hi < hi || t.all_lo > lo) &&
        workgroup_any(fabsf(l) < INFINITY && not_finite<D / 16>(acc), smem)) {
      only = t.i0;
      continue;
    }

    write_rows16<D, NW>(a, c, it, t, smem, wv, n, g4, acc, m, l, only);
    if (only < 0 || ++only > t.i1) return;
    __syncthreads();
  }
}

// ------------------------------------------------------------------ many rows
// Tiles of 32 RG rows.  A wave holds 32 rows and RG waves share the staged
// keys; KG = 4 / RG such groups take the 32-key steps of the piece in turn.
// Two workgroups a CU: one's matrix products run under the other's softmax.
//
// The products for the scores of step i + 1 come before the softmax of step i,
// so that the matrix cores work while rows are staged and maxima taken: K is
// wanted one step before V, and their two rings in LDS are NB steps deep each.
//
// A prompt of 2048 (64 heads of 128) takes 84 us, 820 TFLOP/s, a chunk of 509
// over 16384 keys in 8 bits 297 us with its join, 934 TFLOP/s; the matrix cores
// are busy 34% and 41% of the time (rocprofv3).  What bounds bf16 is the latency
// of a wave's step: one workgroup a CU takes twice the time, and of its parts,
// left out one at a time, the staging gives 14%, the exponentials, the reads of K
// or V, the look or the barrier 5% at most.  In 8 bits the staging is the largest
// part: without its loads, conversions and writes to LDS a step is 23% shorter.
// The registers (64 sums, 32 of Q, 32 scores a lane) allow two waves a SIMD.
//
// bf16 rows go straight from memory to LDS.  e4m3 rows pass through registers
// and are written as bf16, each times its scale (exact), so that the
// conversion is made once for the workgroup and not by every wave.
template <int D, bool Q8, int RG>
struct Many {
  static constexpr int KG = 4 / RG, R = 32 * RG;
  static constexpr int NB = Q8 || RG == 2 ? 2 : 4;
  static constexpr int AHEAD = RG == 4 ? 2 : 1;      // e4m3: steps in registers
  static constexpr int ROWB = 2 * D;                 // in LDS
  static constexpr int STAGE = 32 * ROWB;            // 32 keys of K or V
  static constexpr int RING = 2 * NB * STAGE;        // K's, then V's
  static constexpr int SUMS = KG > 1 ? KG * R * (D + 2) * 4 : 0;
  static constexpr int SMEM = KG * RING > SUMS ? KG * RING : SUMS;
};

template <int I>
using Step = std::integral_constant<int, I>;

template <int D, bool Q8, int RG>
__global__ __launch_bounds__(256, 2) void attend_many_kernel(const AttnArgs a, const Cut c) {
  using M = Many<D, Q8, RG>;
  constexpr int KG = M::KG, R = M::R, NB = M::NB, ROWB = M::ROWB, STAGE = M::STAGE;
  constexpr int AHEAD = M::AHEAD;
  constexpr int SRC = Q8 ? D : 2 * D;                // bytes of a row in memory
  constexpr int P = SRC / 16;                        // its 16-byte pieces
  constexpr int KPI = 64 / P;                        // keys per load of a wave
  constexpr int LOADS = 32 / KPI;                    // loads per step of K, over RG waves
  constexpr int MINE = (LOADS + RG - 1) / RG;        // at most, by one wave
  // One workgroup's matrix products go first and the other's softmax fills in:
  // with it / without, a prompt of 2048 84.4 / 86.7 us, in 8 bits 87.9 / 93.7, of
  // 64 dims 51.8 / 54.1.  Not for e4m3 rows of 64 dims, where a step has as much
  // conversion as products, and those wait for it (64.4 / 53.5, 8192 tokens 765 /
  // 647).
  constexpr bool FIRST = !Q8 || D == 128;
  __shared__ __attribute__((aligned(16))) char smem[M::SMEM];

  Item it;
  if (!find_item<false>(a, c, a.first + (int)blockIdx.x, it)) return;
  const int lane = threadIdx.x & 63;
  const int wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int rg = wv % RG, kg = wv / RG;
  const int n = lane & 31, hh = lane >> 5;
  const Tile t = tile_of(a, it.q0, it.n, it.len, it.tile, R);
  int lo, hi, kbeg, steps, vis_hi, all_hi;   // of a pass

  // Q^T of the wave's rows and what each of them sees
  u32x4 qf[D / 16];
  const int my = t.row0 + min(32 * rg + n, t.rows - 1);
  const int qi = a.by_group.of(my);
  const uint16_t* qp = a.q + (int64_t)(t.first_q + qi) * a.q_token_stride +
                       (int64_t)(it.head * a.group + my - qi * a.group) * a.q_head_stride;
#pragma unroll
  for (int s = 0; s < D / 16; ++s)
    qf[s] = *reinterpret_cast<const u32x4_any*>(qp + 16 * s + 8 * hh);
  const int vis_lo = a.window ? t.pos0 + qi - a.window + 1 : 0;
  // the first and last query of the wave's rows: keys that all of them see
  const int first_q = a.by_group.of(t.row0 + min(32 * rg, t.rows - 1));
  const int last_q = a.by_group.of(t.row0 + min(32 * rg + 31, t.rows - 1));
  const int all_lo =
      __builtin_amdgcn_readfirstlane(a.window ? t.pos0 + last_q - a.window + 1 : 0);

  char* kring = smem + kg * M::RING;
  char* vring = kring + NB * STAGE;
  bool bad = false;
  int blocks = -1;   // lane 2 i + h: rows / 16 of the cache for half h of step i (mod 32)

  auto find_blocks = [&](int i) {
    const int64_t key = (int64_t)kbeg + (int64_t)32 * KG * (i + (lane >> 1)) + 16 * (lane & 1);
    blocks = -1;
    if (key < hi) {
      const int at = a.by_page.of((int)key);
      const int page = a.table[(int64_t)it.b * a.width + at];
      if (page >= 0 && page < a.pages)
        blocks =
            (int)((((int64_t)page * a.kv_heads + it.head) * a.page + (key - at * a.page)) >> 4);
      else  // a page that the cache lacks: the rows that see it are NaN
        bad |= key + 16 > lo;
    }
  };
  // A wave's share of a step lies in one half of it: rows / 16 of the half and
  // its valid keys, [below, keys).
  const int half = MINE * rg / (LOADS / 2) & 1;
  struct Rows {
    int blk, keys, below;
  };
  auto rows_of = [&](int i) {
    if ((i & 31) == 0) find_blocks(i);
    Rows r;
    const int key0 = kbeg + 32 * KG * i + 16 * half;
    const int blk = __builtin_amdgcn_readlane(blocks, 2 * (i & 31) + half);
    // the same for the whole wave, which the compiler cannot see of all of it
    r.below = __builtin_amdgcn_readfirstlane(lo - key0);
    r.keys = __builtin_amdgcn_readfirstlane(
        blk < 0 || i >= steps ? 0 : min(max(hi - key0, 0), 16));
    r.blk = __builtin_amdgcn_readfirstlane(max(blk, 0));
    return r;
  };

  // bf16: the wave's share of a step of K (w = 0) or V (1), straight into LDS
  auto stage = [&](int w, int at, const Rows& r) {
    char* st = (w ? vring : kring) + at * STAGE;
    const uint8_t* src = a.cache[w] + (int64_t)r.blk * (16 * SRC);
#pragma unroll
    for (int j = 0; j < MINE; ++j) {
      const int load = MINE * rg + j;                // of the step's LOADS
      const int key = (load % (LOADS / 2)) * KPI + lane / P;   // of the half
      const int off = key * SRC + (((lane % P) ^ swizzle<ROWB>(key)) << 4);
      lds_bload16(src, r.keys * SRC, key < r.below ? 1 << 30 : off, 0, st + load * 1024);
    }
  };
  // e4m3: the same rows and their scales into registers, then as bf16 into LDS
  u32x4 raw[AHEAD][2][MINE];
  uint32_t sc[AHEAD][2][MINE];
  auto fetch = [&](int w, int slot, const Rows& r) {
    if (LOADS < RG * MINE && MINE * rg >= LOADS) return;
    const int64_t at = (int64_t)r.blk * 16;
#pragma unroll
    for (int j = 0; j < MINE; ++j) {
      const int key = ((MINE * rg + j) % (LOADS / 2)) * KPI + lane / P;
      const bool below = key < r.below;
      raw[slot][w][j] = bload128(a.cache[w] + at * SRC, r.keys * SRC,
                                 below ? 1 << 30 : key * SRC + (lane % P) * 16, 0);
      sc[slot][w][j] = bload8(a.scale[w] + at, r.keys, below ? 1 << 30 : key, 0);
    }
  };
  auto put = [&](int w, int slot, int at) {
    if (LOADS < RG * MINE && MINE * rg >= LOADS) return;
    char* st = (w ? vring : kring) + at * STAGE;
#pragma unroll
    for (int j = 0; j < MINE; ++j) {
      const int key = (MINE * rg + j) * KPI + lane / P;   // of the step
      const float s = __uint_as_float(sc[slot][w][j] << 23);
      const u32x4 got = raw[slot][w][j];
      // A lane has two neighbouring pieces of 16 bytes.  Every other four lanes
      // write theirs in opposite order, so that eight lanes write to all banks:
      // half of the conflicts, a chunk of 509 over 16384 keys 296 / 300 us.  For
      // 64 dims the exchange costs more (16000 tokens of 16 heads 635 / 623 us).
      const bool swap = D == 128 && (lane & 4);
      const u32x4 r = {swap ? got[2] : got[0], swap ? got[3] : got[1], swap ? got[0] : got[2],
                       swap ? got[1] : got[3]};
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int piece = 2 * (lane % P) + (e ^ (int)swap);
        *reinterpret_cast<u32x4*>(st + key * ROWB + ((piece ^ swizzle<ROWB>(key)) << 4)) =
            u32x4{bf16x2_of_e4m3<false>(r[2 * e], s), bf16x2_of_e4m3<true>(r[2 * e], s),
                  bf16x2_of_e4m3<false>(r[2 * e + 1], s), bf16x2_of_e4m3<true>(r[2 * e + 1], s)};
      }
    }
  };

  f32x16 acc[D / 32], nil;
#pragma unroll
  for (int r = 0; r < 16; ++r) nil[r] = 0.f;
  float m, l;

  // sixteen dims of K of a stage
  auto keys = [&](int at, int s) {
    return *reinterpret_cast<const u32x4*>(
        kring + at * STAGE + n * ROWB + (((2 * s + hh) ^ swizzle<ROWB>(n)) << 4));
  };

  // Masks the scores of step i and moves the references.
  auto look = [&](int i, f32x16& z) {
    const int key0 = kbeg + 32 * KG * i;
    if (key0 + 32 > all_hi || key0 < all_lo) {
#pragma unroll
      for (int r = 0; r < 16; ++r) {
        const int j = key0 + 8 * (r >> 2) + 4 * hh + (r & 3);
        z[r] = j < vis_hi && j >= vis_lo ? z[r] : -INFINITY;
      }
    }
    float top = z[0];
#pragma unroll
    for (int r = 1; r < 16; ++r) top = fmaxf(top, z[r]);
    top *= a.scale_log2;
    // only when a score passes the reference by 2^6: see above
    if (__ballot(top > m + 6.f)) {
      top = fmaxf(top, __shfl_xor(top, 32));
      const float m1 = fmaxf(m, top);
      const float f = m1 == -INFINITY ? 1.f : __builtin_amdgcn_exp2f(m - m1);
      m = m1;
      l *= f;
#pragma unroll
      for (int d = 0; d < D / 32; ++d) acc[d] *= f;
    }
  };

  // Two scores to packed weights: pf[c] holds the keys 16 c + 8 (j / 4) +
  // 4 hh + j % 4 of the step.
  auto weigh = [&](int r, float ref, f32x16& z, u32x4 (&pf)[2]) {
    const float p0 = __builtin_amdgcn_exp2f(fmaf(z[r], a.scale_log2, -ref));
    const float p1 = __builtin_amdgcn_exp2f(fmaf(z[r + 1], a.scale_log2, -ref));
    pf[r >> 3][(r & 7) >> 1] = weights(p0, p1, l);
  };

  // V^T: lane (dim, hh) of tile d wants the rows 16 c + 4 hh + 0..3 and those
  // + 8; its 16 lanes read them at 4 rows x 32 bytes
  char* voff[D / 32][2];
#pragma unroll
  for (int d = 0; d < D / 32; ++d)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int k = 8 * e + 4 * hh + ((lane & 15) >> 2);
      const int piece = 4 * d + 2 * ((lane >> 4) & 1) + ((lane >> 1) & 1);
      voff[d][e] = vring + k * ROWB + ((piece ^ swizzle<ROWB>(k)) << 4) +
                   8 * (lane & 1);
    }
  auto values = [&](auto at, const u32x4 (&pf)[2]) {
#pragma unroll
    for (int d = 0; d < D / 32; d += 2) {
      u32x4 vf[4];
#pragma unroll
      for (int x = 0; x < 4; ++x)
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          const u32x2 r = read_tr16(voff[d + (x >> 1)][x & 1] + at * STAGE + c * 16 * ROWB);
          vf[(x & 2) + c][2 * (x & 1)] = r[0];
          vf[(x & 2) + c][2 * (x & 1) + 1] = r[1];
        }
#pragma unroll
      for (int k = 0; k < 2; ++k)
#pragma unroll
        for (int e = 0; e < 2; ++e) acc[d + e] = mfma32(vf[2 * e + k], pf[k], acc[d + e]);
    }
  };

  auto meet = [&]() {   // the group's waves: stages written, or read to the end
    if (RG > 1) asm volatile("s_barrier" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
  };

  int only = -1;   // the query of this pass, or all
  for (;;) {
    piece_range(t, it.piece, it.pieces, lo, hi);
    if (only >= 0) query_range(a, t, only, lo, hi);
    lo = __builtin_amdgcn_readfirstlane(lo);
    hi = __builtin_amdgcn_readfirstlane(hi);
    kbeg = (lo & ~31) + 32 * kg;
    steps = __builtin_amdgcn_readfirstlane(
        hi > lo ? (hi - (lo & ~31) + 32 * KG - 1) / (32 * KG) : 0);   // of every group
    vis_hi = min(t.pos0 + qi + 1, hi);
    all_hi = __builtin_amdgcn_readfirstlane(min(t.pos0 + first_q + 1, hi));
#pragma unroll
    for (int d = 0; d < D / 32; ++d)
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[d][r] = 0.f;
    m = -INFINITY;
    l = 0.f;
    if (steps > 0) {
      f32x16 z[2];
      Rows last, coming;   // of the steps that V and K are staged of next
#pragma unroll
      for (int i = 0; i < NB; ++i) {   // K of steps 0 .. NB - 1, V of 0 .. NB - 2
        last = rows_of(i);
        if (Q8) {
          fetch(0, 0, last);
          put(0, 0, i);
        } else {
          stage(0, i, last);
        }
        if (i == NB - 1) break;
        if (Q8) {
          fetch(1, 0, last);
          put(1, 0, i);
        } else {
          stage(1, i, last);
        }
      }
      coming = rows_of(NB);
      if (Q8) {   // in registers: V of AHEAD steps from NB - 1 on, K from NB on
#pragma unroll
        for (int k = 0; k < AHEAD; ++k) {
          fetch(1, (NB - 1 + k) % AHEAD, last);
          fetch(0, (NB + k) % AHEAD, coming);
          last = coming;
          coming = rows_of(NB + k + 1);
        }
      } else {
        wait_loads<0>();
      }
      wait_lds();
      meet();
      z[0] = nil;
#pragma unroll
      for (int s = 0; s < D / 16; ++s) z[0] = mfma32(keys(0, s), qf[s], z[0]);
      // step i = u (mod NB): its scores are in now, those of i + 1 go to next
      auto turn = [&](auto u, int i, f32x16& now, f32x16& next) {
        // K of step i + 1 and V of step i have arrived, and all waves have the
        // scores of step i and the values of step i - 1 behind them: K's stage
        // i and V's stage i - 1 may be written.
        if (!Q8) wait_loads<(NB - 2) * 2 * MINE>();
        wait_lds();
        meet();
        u32x4 kf[D / 16];
#pragma unroll
        for (int s = 0; s < D / 16; ++s) kf[s] = keys((u + 1) % NB, s);
        if (FIRST) __builtin_amdgcn_s_setprio(1);
        next = nil;
#pragma unroll
        for (int s = 0; s < D / 16; ++s) next = mfma32(kf[s], qf[s], next);
        if (Q8) {
          put(0, u % AHEAD, u);
          put(1, (u + NB - 1) % AHEAD, (u + NB - 1) % NB);
          fetch(1, (u + NB - 1) % AHEAD, last);
          fetch(0, u % AHEAD, coming);
        } else {
          stage(1, (u + NB - 1) % NB, last);
          stage(0, u, coming);
        }
        if (FIRST) __builtin_amdgcn_s_setprio(0);
        look(i, now);
        const float ref = m == -INFINITY ? 0.f : m;
        u32x4 pf[2];
#pragma unroll
        for (int r = 0; r < 16; r += 2) weigh(r, ref, now, pf);
        if (FIRST) __builtin_amdgcn_s_setprio(1);
        values(u, pf);
        if (FIRST) __builtin_amdgcn_s_setprio(0);
        last = coming;
        coming = rows_of(i + NB + 1 + (Q8 ? AHEAD : 0));
      };
      for (int i = 0; i < steps; i += NB) {
        turn(Step<0>{}, i, z[0], z[1]);
        // a turn past the last step finds no keys; without a branch here the
        // rows on their way through registers need not arrive for a copy
        if (Q8 || i + 1 < steps) turn(Step<1>{}, i + 1, z[1], z[0]);
        if constexpr (NB == 4) {
          if (i + 2 < steps) turn(Step<2>{}, i + 2, z[0], z[1]);
          if (i + 3 < steps) turn(Step<3>{}, i + 3, z[1], z[0]);
        }
      }
    }
    wait_loads<0>();
    wait_lds();
    if (__ballot(bad)) l = NAN;
    l += __shfl_xor(l, 32);
    if (only < 0 && (t.all_hi < hi || t.all_lo > lo) &&
        workgroup_any(fabsf(l) < INFINITY && not_finite<D / 32>(acc), smem)) {
      only = t.i0;
      continue;
    }

    write_many<D, RG>(a, c, it, t, smem, rg, kg, n, hh, my, qi, acc, m, l, only);
    if (only < 0 || ++only > t.i1) return;
    __syncthreads();
  }
}

template <int D, bool Q8>
hipError_t run(const AttnArgs& a, hipStream_t s) {
  // Waves of a workgroup of few rows: two rings of 64 KB at most fit a CU, and
  // then the second workgroup's start and end lie under the first one's loads.
  // bf16 rows of 128 dims with 2 / 4 waves: a token at 4097 keys 14.2 / 13.9
  // us, 4 of them 22.7 / 27.4, 32 sequences of up to 16000 keys 152 / 156.
  constexpr int NW = !Q8 && D == 128 ? 2 : 4;
  return run_cuts<D>(a, NW * 64, s, [&](const AttnArgs& b, const Cut& c, unsigned grid) {
    if (c.R == 16)
      attend_rows16_kernel<D, Q8, NW, 2><<<grid, NW * 64, 0, s>>>(b, c);
    else if (c.R == 64)
      attend_many_kernel<D, Q8, 2><<<grid, 256, 0, s>>>(b, c);
    else
      attend_many_kernel<D, Q8, 4><<<grid, 256, 0, s>>>(b, c);
  });
}

}  // namespace

Divisor divisor(int by) {
  Divisor d{1, 0, by};
  while ((int64_t(1) << d.shift) < by) ++d.shift;
  d.mul = (uint32_t)(((uint64_t(1) << 32) * ((uint64_t(1) << d.shift) - by)) / by + 1);
  return d;
}

size_t paged_attention_workspace(const AttnArgs& a) {
  return way_bytes(way_of_size(a));
}

hipError_t launch_paged_attention(const AttnArgs& a, hipStream_t s) {
  if (a.bits == 4) return launch_attention_4bit(a, s);
  const bool q8 = a.bits == 8;
  if (a.dim == 64) return q8 ? run<64, true>(a, s) : run<64, false>(a, s);
  return q8 ? run<128, true>(a, s) : run<128, false>(a, s);
}

}  // namespace bd
