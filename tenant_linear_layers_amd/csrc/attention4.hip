// Attention of new tokens over a paged key/value cache in e2m1 with an e8m0
// scale per 32 dims; the definition and the plan are in attention_plan.h.
//
// Scores.  A lane converts its part of K in registers (e2m1 times a power of two is
// a bf16 number), and the products are those of a bf16 cache, exact and summed in
// float32.  Over many rows the scaled matrix instructions would take K as it is
// stored, with a row of q as two parts of e4m3, in the same time on the matrix cores
// and without the conversion, 32 vector instructions a step and wave (a chunk of 509
// over 16384 keys 266 us for 293, a prompt of 2048 85 for 89, mixed calls 0 to 5%
// less).  But they keep a product to about 17 bits below the largest of its group: with
// one dim of q at 512 or 1024 against keys of 4 the output's error was 0.012 to 0.017
// and 0.030 to 0.043; it is 0.0018 with exact ones, the roundings' own.
//
// Values.  The product with V runs over the keys, whose scales differ, so V is
// converted everywhere.  A lane converts up to 16 bytes of a group by the
// instruction that takes its scale, writes them to LDS as bf16, and they are read
// back transposed.
#include <type_traits>

#include "attention_plan.h"
#include "common.h"
#include "e2m1.h"
#include "layer.h"

namespace bd {
namespace {

// N dwords at an address aligned to all of them.
template <int N>
__device__ __forceinline__ void load_dwords(const uint8_t* p, uint32_t (&v)[N]) {
  if constexpr (N == 4) {
    const u32x4 x = ld128(p);
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = x[i];
  } else if constexpr (N == 2) {
    const u32x2 x = *reinterpret_cast<const u32x2*>(p);
    v[0] = x[0];
    v[1] = x[1];
  } else {
    v[0] = ld32(p);
  }
}

__device__ __forceinline__ u32x4 load_past(const uint8_t* p) {   // not to stay in the caches
  return __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(p));
}

// Four blocks of four rows, 32 bytes apart from AT on, and those NEXT bytes
// behind each; the wait is in the statement.
template <int AT, int NEXT>
__device__ __forceinline__ void read_tr16_4(uint32_t at, u32x4 (&v)[4]) {
  u32x2 r[8];
  asm volatile(
      "ds_read_b64_tr_b16 %0, %8 offset:%9\n"
      "ds_read_b64_tr_b16 %1, %8 offset:%10\n"
      "ds_read_b64_tr_b16 %2, %8 offset:%11\n"
      "ds_read_b64_tr_b16 %3, %8 offset:%12\n"
      "ds_read_b64_tr_b16 %4, %8 offset:%13\n"
      "ds_read_b64_tr_b16 %5, %8 offset:%14\n"
      "ds_read_b64_tr_b16 %6, %8 offset:%15\n"
      "ds_read_b64_tr_b16 %7, %8 offset:%16\n"
      "s_waitcnt lgkmcnt(0)"
      : "=&v"(r[0]), "=&v"(r[1]), "=&v"(r[2]), "=&v"(r[3]), "=&v"(r[4]), "=&v"(r[5]),
        "=&v"(r[6]), "=&v"(r[7])
      : "v"(at), "n"(AT), "n"(AT + NEXT), "n"(AT + 32), "n"(AT + 32 + NEXT), "n"(AT + 64),
        "n"(AT + 64 + NEXT), "n"(AT + 96), "n"(AT + 96 + NEXT)
      : "memory");
#pragma unroll
  for (int i = 0; i < 4; ++i)
    v[i] = u32x4{r[2 * i][0], r[2 * i][1], r[2 * i + 1][0], r[2 * i + 1][1]};
}

// ------------------------------------------------------------------ few rows
// Tiles of 16 rows.  The NW waves of a workgroup take 32-key steps of the piece
// in turn, each with its own stage of V in LDS, so there is no barrier until
// the waves' sums are joined.  Rows go from memory to registers a step ahead: a
// step's 32 rows are two runs of 16, each contiguous in its page, and a lane's
// bytes are an operand of K, or a group of V, as they lie there.
//
// Bound by HBM: 32 sequences of 8000 keys (279 MB) 57 us with their join, 4.9 TB/s
// (a copy reaches 5.2), 64 of 1000 to 16000 (364 to 395 MB as they are drawn) 82 to
// 91 by card.  A single token at 4097 keys, 8.3 us, is a chain of latencies.  Three
// workgroups a CU for 128 dims, 168 registers a lane: for four 42 spill.
template <int D, int NW>
struct Few4 {
  // V in LDS: rows 32 bytes apart in the banks, so that the eight rows of a
  // transposing read lie in different ones, and every place is a lane's own plus
  // a constant.
  static constexpr int R = 16, ROWL = 2 * D + 32, STAGE = 32 * ROWL;
  static constexpr int SUMS = NW * R * (D + 2) * 4;
  static constexpr int SMEM = NW * STAGE > SUMS ? NW * STAGE : SUMS;
};

template <int D, int NW>
__device__ __forceinline__ void attend4_rows16(const AttnArgs& a, const Cut& c, int item,
                                               char* smem) {
  using F = Few4<D, NW>;
  constexpr int R = F::R, ROWL = F::ROWL, STAGE = F::STAGE;
  constexpr int ROWB = D / 2, GROUPS = D / kGroup4;   // bytes, scales of a row
  constexpr int VLOADS = D / 64;                      // 16 bytes a lane: 32 rows of V
  constexpr int KD = D / 4;                           // dims of K a lane and key

  Item it;
  if (!find_item<false>(a, c, item, it)) return;
  const int lane = threadIdx.x & 63;
  const int wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int n = lane & 15, g4 = lane >> 4;
  const Tile t = tile_of(a, it.q0, it.n, it.len, it.tile, R);
  int lo, hi, kbeg, steps, vis_hi;   // of a pass

  // Q^T: lane n's row, the KD dims that the lane's piece of K holds.
  const int my = min(n, t.rows - 1);
  const int qi = a.by_group.of(t.row0 + my);
  const uint16_t* qp =
      a.q + (int64_t)(t.first_q + qi) * a.q_token_stride +
      (int64_t)(it.head * a.group + (t.row0 + my) - qi * a.group) * a.q_head_stride;
  u32x4 qf[KD / 8];
#pragma unroll
  for (int s = 0; s < KD / 8; ++s)
    qf[s] = *reinterpret_cast<const u32x4_any*>(qp + KD * g4 + 8 * s);
  const int pos = t.pos0 + qi;
  const int vis_lo = a.window ? pos - a.window + 1 : 0;

  char* vst = smem + wv * STAGE;
  bool bad = false;
  int blocks = -1;   // lane 2 i + h: rows / 16 of the cache for half h of step i (mod 32)
  const int vpiece = lane % GROUPS;                    // V's group of the lane
  const int vkey = lane / GROUPS;                      // and its row, of the first load
  // its bytes of 16 rows of K and of V, and the group of its dims of K
  const uint32_t koff = n * ROWB + g4 * (KD / 2), voff = lane % (16 * GROUPS) * 16;
  const int kgroup = g4 * KD / kGroup4;
  char* vput = vst + vkey * ROWL + vpiece * 64;
  const uint32_t vget =
      lds_address(vst + (4 * g4 + (n >> 2)) * ROWL + ((n >> 1) & 1) * 16 + 8 * (n & 1));

  // V's rows, whole lines by a load, are read past the caches' turn of use: K's,
  // whose lines several parts of a load want, stay longer (64 sequences of up to
  // 16000 keys 86 us, both so 94, neither 102; 4 of 4097 keys 16.0, 14.5 and 15.7).
  // A step's scales come with one load, of K's rows to lanes 0..31 and of V's to
  // the others, and go from there to the lanes that want them: loads of their
  // own for every operand take 4 us of 80 (40 sequences of 8000 keys).
  const uint8_t* sbase = lane < 32 ? a.scale[0] : a.scale[1];
  struct Rows {
    uint32_t k[2][KD / 8];
    u32x4 v[VLOADS];
    uint32_t sc;
  };
  auto fetch = [&](int i, Rows& r) {
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
    // halves that are not there are read from block 0
    int blk[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      blk[h] = max(__builtin_amdgcn_readlane(blocks, 2 * (i & 31) + h), 0);
      const int64_t row = (int64_t)blk[h] * (16 * ROWB);
      load_dwords<KD / 8>(a.cache[0] + row + koff, r.k[h]);
      if (D == 128) r.v[h % VLOADS] = load_past(a.cache[1] + row + voff);
    }
    if (D == 64)   // a half of the lanes each
      r.v[0] = load_past(a.cache[1] + (int64_t)(lane < 32 ? blk[0] : blk[1]) * (16 * ROWB) + voff);
    const uint8_t* sp =
        sbase + (int64_t)(lane & 16 ? blk[1] : blk[0]) * (16 * GROUPS) + (lane & 15) * GROUPS;
    r.sc = D == 128 ? ld32(sp) : *reinterpret_cast<const uint16_t*>(sp);
    __builtin_amdgcn_sched_barrier(0);   // on their way before a step waits for its own
  };

  f32x4 acc[D / 16];
  float m, l;

  auto step = [&](int i, const Rows& r) {
    const int key0 = kbeg + 32 * NW * i;
    const bool ends = key0 < lo || key0 + 32 > hi;   // rows of it do not count
    uint32_t ks[2], vs[VLOADS];
#pragma unroll
    for (int h = 0; h < 2; ++h)
      ks[h] = (uint32_t)__shfl((int)r.sc, 16 * h + n) >> (8 * kgroup) & 0xFFu;
#pragma unroll
    for (int h = 0; h < VLOADS; ++h)
      vs[h] = (uint32_t)__shfl((int)r.sc, 32 + 16 * h + vkey) >> (8 * vpiece) & 0xFFu;
    float s[8];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      f32x4 z = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int p = 0; p < KD / 8; ++p)
        z = mfma16(bf16x8_of_e2m1(r.k[h][p], __uint_as_float(ks[h] << 23)), qf[p], z);
#pragma unroll
      for (int e = 0; e < 4; ++e) s[4 * h + e] = z[e];
    }
    if (ends) {   // the smallest scale: finite under their weights of zero
      asm volatile("");   // a branch, not comparisons in every step
#pragma unroll
      for (int h = 0; h < VLOADS; ++h) {
        const int key = key0 + 16 * h + vkey;
        vs[h] = key >= lo && key < hi ? vs[h] : 0u;
      }
    }
    // V as bf16 into LDS
#pragma unroll
    for (int h = 0; h < VLOADS; ++h) {
      const float sc = __uint_as_float(vs[h] << 23);
#pragma unroll
      for (int j = 0; j < 4; ++j)
        *reinterpret_cast<u32x4*>(vput + 16 * h * ROWL + 16 * j) = bf16x8_of_e2m1(r.v[h][j], sc);
    }
    // a mask only where some row of the tile sees part of the step
    if (ends || key0 + 32 > t.all_hi || key0 < t.all_lo) {
      asm volatile("");
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int j = key0 + 16 * (e >> 2) + 4 * g4 + (e & 3);
        s[e] = j < vis_hi && j >= max(vis_lo, lo) ? s[e] : -INFINITY;
      }
    }
    float top = s[0];
#pragma unroll
    for (int e = 1; e < 8; ++e) top = fmaxf(top, s[e]);
    top *= a.scale_log2;
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
    for (int e = 0; e < 8; e += 2)
      pf[e >> 1] = weights(__builtin_amdgcn_exp2f(fmaf(s[e], a.scale_log2, -ref)),
                           __builtin_amdgcn_exp2f(fmaf(s[e + 1], a.scale_log2, -ref)), l);
    u32x4 vf[4];   // of four tiles of 16 dims
    read_tr16_4<0, 16 * ROWL>(vget, vf);
#pragma unroll
    for (int e = 0; e < 4; ++e) acc[e] = mfma16(vf[e], pf, acc[e]);
    if constexpr (D == 128) {
      read_tr16_4<128, 16 * ROWL>(vget, vf);
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[4 + e] = mfma16(vf[e], pf, acc[4 + e]);
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
      Rows r[2];
      fetch(0, r[0]);
      for (int i = 0; i < steps; i += 2) {
        // past the last step there are no rows left to count: with a branch here a
        // step would have to wait for the next one's loads
        fetch(i + 1, r[1]);
        step(i, r[0]);
        fetch(i + 2, r[0]);
        if (i + 1 < steps) step(i + 1, r[1]);
      }
    }
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
// Rows pass through registers; K is written to LDS as it is and converted by each
// wave for its products (as bf16 it would be four times the reads of LDS), V as bf16,
// each group times its scale, so that the conversion is made once for the workgroup.
//
// A chunk of 509 over 16384 keys (64 heads of 128) takes 291 to 293 us with its
// join, 950 TFLOP/s (a library product 1324; over 8 bits 300), a prompt of 2048 88
// to 95 us by card.  The matrix cores are busy 41% of the time, the vector ALU 49%
// (168 instructions a step beside 16 products, 32 of them K's conversion, 32 the
// exponentials and their arguments): with two waves a SIMD, as many as 226 registers
// allow, there is little of either left.
template <int D, int RG>
struct Many4 {
  static constexpr int KG = 4 / RG, R = 32 * RG;
  static constexpr int NB = 2;
  static constexpr int AHEAD = RG == 4 ? 2 : 1;      // steps in registers
  // Bytes of a row, and of one of K and V in LDS: K's 16 bytes and V's 64 apart
  // in the banks, for reads of a piece of many rows and of 64 bytes of four.
  static constexpr int ROW = D / 2, ROWK = ROW + 16, ROWV = 2 * D + 64;
  static constexpr int STAGEK = 32 * ROWK, STAGEV = 32 * ROWV;
  static constexpr int SCALES = 32 * (D / kGroup4);     // K's of a step
  static constexpr int RING = NB * (STAGEK + STAGEV + SCALES);   // K's, V's, scales
  static constexpr int SUMS = KG > 1 ? KG * R * (D + 2) * 4 : 0;
  static constexpr int SMEM = KG * RING > SUMS ? KG * RING : SUMS;
};

template <int I>
using Step = std::integral_constant<int, I>;

// N dwords to a place in LDS aligned to all of them.
template <int N>
__device__ __forceinline__ void store_dwords(char* p, const uint32_t (&v)[N]) {
  if constexpr (N == 4) *reinterpret_cast<u32x4*>(p) = u32x4{v[0], v[1], v[2], v[3]};
  else if constexpr (N == 2) *reinterpret_cast<u32x2*>(p) = u32x2{v[0], v[1]};
  else *reinterpret_cast<uint32_t*>(p) = v[0];
}
template <int D, int RG>
__device__ __forceinline__ void attend4_many(const AttnArgs& a, const Cut& c, int item,
                                             char* smem) {
  using M = Many4<D, RG>;
  constexpr int KG = M::KG, R = M::R, NB = M::NB, ROW = M::ROW, ROWK = M::ROWK, ROWV = M::ROWV;
  constexpr int AHEAD = M::AHEAD, GROUPS = D / kGroup4;
  constexpr int W = 32 * ROW / (RG * 64 * 4);        // dwords of a step's K a lane
  constexpr int LPR = ROW / (4 * W);                 // lanes a row
  constexpr int MINE = 64 / LPR;                     // rows of a step, by one wave
  // One workgroup's matrix products go first and the other's softmax fills in.
  // Not for tiles of 64 rows of 64 dims (24 mixed sequences 43.4 us, with it 44.1; a
  // prompt of 2048 in tiles of 128 55.5 and 52.1).
  constexpr bool FIRST = D == 128 || RG == 4;

  Item it;
  if (!find_item<false>(a, c, item, it)) return;
  const int lane = threadIdx.x & 63;
  const int wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int rg = wv % RG, kg = wv / RG;
  const int n = lane & 31, hh = lane >> 5;
  const Tile t = tile_of(a, it.q0, it.n, it.len, it.tile, R);
  int lo, hi, kbeg, steps, vis_hi, all_hi;   // of a pass

  // Q^T of the wave's rows, for 64 dims at a time those of 16 hh .. + 15 and
  // 32 + 16 hh .. + 15, and what each row sees
  const int my = t.row0 + min(32 * rg + n, t.rows - 1);
  const int qi = a.by_group.of(my);
  const uint16_t* qp = a.q + (int64_t)(t.first_q + qi) * a.q_token_stride +
                       (int64_t)(it.head * a.group + my - qi * a.group) * a.q_head_stride;
  u32x4 qf[D / 16];
#pragma unroll
  for (int e = 0; e < D / 16; ++e)
    qf[e] = *reinterpret_cast<const u32x4_any*>(qp + 64 * (e >> 2) + 32 * hh + 8 * (e & 3));
  const int vis_lo = a.window ? t.pos0 + qi - a.window + 1 : 0;
  // the first and last query of the wave's rows: keys that all of them see
  const int first_q = a.by_group.of(t.row0 + min(32 * rg, t.rows - 1));
  const int last_q = a.by_group.of(t.row0 + min(32 * rg + 31, t.rows - 1));
  const int all_lo =
      __builtin_amdgcn_readfirstlane(a.window ? t.pos0 + last_q - a.window + 1 : 0);

  char* kring = smem + kg * M::RING;
  char* vring = kring + NB * M::STAGEK;
  char* sring = vring + NB * M::STAGEV;
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
  // A wave's share of a step lies in one half of it: rows / 16 of it and
  // its valid keys, [below, keys).  Rows that are not there are read
  // from block 0 and count for nothing.
  const int half = MINE * rg / 16;
  struct Rows {
    int blk, keys, below;
  };
  auto rows_of = [&](int i) {
    if ((i & 31) == 0) find_blocks(i);
    Rows r;
    const int key0 = kbeg + 32 * KG * i + 16 * half;
    const int blk = __builtin_amdgcn_readlane(blocks, 2 * (i & 31) + half);
    // the same for the whole wave, which the compiler cannot see of all of it
    r.keys = __builtin_amdgcn_readfirstlane(
        blk < 0 || i >= steps ? 0 : min(max(hi - key0, 0), 16));
    r.blk = __builtin_amdgcn_readfirstlane(max(blk, 0));
    r.below = __builtin_amdgcn_readfirstlane(lo - key0);
    return r;
  };

  // A wave's rows of a step of K (w = 0) or V (1) into registers, then into LDS.
  // Scales of rows that do not count are 0, 2^-127: V is finite under a weight of
  // zero.
  const int row = MINE * rg + lane / LPR;              // of the step
  const int dword = lane % LPR * W;                    // of the row
  char* kput = kring + row * ROWK + dword * 4;
  char* vput = vring + row * ROWV + dword * 16;
  char* sput = sring + row * GROUPS + dword / 4;
  uint32_t raw[AHEAD][2][W], sc[AHEAD][2];
  auto fetch = [&](int w, int slot, const Rows& r) {
    const int64_t at = (int64_t)r.blk * 16;
    const int key = row & 15;
    load_dwords<W>(a.cache[w] + (at + key) * ROW + dword * 4, raw[slot][w]);
    sc[slot][w] = bload8(a.scale[w] + at * GROUPS, r.keys * GROUPS,
                         key < r.below ? 1 << 30 : key * GROUPS + dword / 4, 0);
  };
  auto put = [&](int w, int slot, int at) {
    if (w == 0) {
      store_dwords<W>(kput + at * M::STAGEK, raw[slot][0]);
      sput[at * M::SCALES] = (char)sc[slot][0];
    } else {
      const float s = __uint_as_float(sc[slot][1] << 23);
#pragma unroll
      for (int j = 0; j < W; ++j)
        *reinterpret_cast<u32x4*>(vput + at * M::STAGEV + 16 * j) =
            bf16x8_of_e2m1(raw[slot][1][j], s);
    }
  };
  // The scales of key n of a stage, byte 2 p that of the lane's 32 dims of the
  // p-th 64.
  auto key_scales = [&](int at) {
    const char* p = sring + at * M::SCALES + n * GROUPS;
    const uint32_t all = D == 128 ? *reinterpret_cast<const uint32_t*>(p)
                                  : *reinterpret_cast<const uint16_t*>(p);
    return all >> (8 * hh);
  };

  f32x16 acc[D / 32], nil;
#pragma unroll
  for (int r = 0; r < 16; ++r) nil[r] = 0.f;
  float m, l;

  // 64 dims of K of a stage
  auto keys = [&](int at, int p) {
    return *reinterpret_cast<const u32x4*>(kring + at * M::STAGEK + n * ROWK + 16 * hh + 32 * p);
  };
  auto scores = [&](const u32x4 (&kf)[D / 64], uint32_t ks) {
    f32x16 z = nil;
#pragma unroll
    for (int p = 0; p < D / 64; ++p) {
      const float sc = __uint_as_float((ks >> (16 * p) & 0xFFu) << 23);
#pragma unroll
      for (int e = 0; e < 4; ++e) z = mfma32(bf16x8_of_e2m1(kf[p][e], sc), qf[4 * p + e], z);
    }
    return z;
  };

  // Masks the scores of step i and moves the references.
  auto look = [&](int i, f32x16& z) {
    const int key0 = kbeg + 32 * KG * i;
    if (key0 + 32 > all_hi || key0 < all_lo || key0 < lo) {
#pragma unroll
      for (int r = 0; r < 16; ++r) {
        const int j = key0 + 8 * (r >> 2) + 4 * hh + (r & 3);
        z[r] = j < vis_hi && j >= max(vis_lo, lo) ? z[r] : -INFINITY;
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
  char* vget = vring + (4 * hh + ((lane & 15) >> 2)) * ROWV + 32 * ((lane >> 4) & 1) +
               16 * ((lane >> 1) & 1) + 8 * (lane & 1);
  auto values = [&](auto at, const u32x4 (&pf)[2]) {
#pragma unroll
    for (int d = 0; d < D / 32; d += 2) {
      u32x4 vf[4];
#pragma unroll
      for (int x = 0; x < 4; ++x)
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          const u32x2 r = read_tr16(vget + at * M::STAGEV + 64 * (d + (x >> 1)) +
                                    (8 * (x & 1) + 16 * c) * ROWV);
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
    asm volatile("s_barrier" ::: "memory");
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
      for (int i = 0; i < NB; ++i) {   // K of steps 0 and 1, V of 0
        last = rows_of(i);
        fetch(0, 0, last);
        put(0, 0, i);
        if (i == NB - 1) break;
        fetch(1, 0, last);
        put(1, 0, i);
      }
      coming = rows_of(NB);
#pragma unroll
      for (int k = 0; k < AHEAD; ++k) {   // in registers: V from step 1 on, K from 2 on
        fetch(1, (NB - 1 + k) % AHEAD, last);
        fetch(0, (NB + k) % AHEAD, coming);
        last = coming;
        coming = rows_of(NB + k + 1);
      }
      wait_lds();
      meet();
      {
        u32x4 kf[D / 64];
#pragma unroll
        for (int p = 0; p < D / 64; ++p) kf[p] = keys(0, p);
        z[0] = scores(kf, key_scales(0));
      }
      // step i = u (mod NB): its scores are in now, those of i + 1 go to next
      auto turn = [&](auto u, int i, f32x16& now, f32x16& next) {
        // K of step i + 1 and V of step i have arrived, and all waves have the
        // scores of step i and the values of step i - 1 behind them: K's stage
        // i and V's stage i - 1 may be written.
        wait_lds();
        meet();
        u32x4 kf[D / 64];
#pragma unroll
        for (int p = 0; p < D / 64; ++p) kf[p] = keys((u + 1) % NB, p);
        const uint32_t ks = key_scales((u + 1) % NB);
        if (FIRST) __builtin_amdgcn_s_setprio(1);
        next = scores(kf, ks);
        put(0, u % AHEAD, u);
        put(1, (u + NB - 1) % AHEAD, (u + NB - 1) % NB);
        fetch(1, (u + NB - 1) % AHEAD, last);
        fetch(0, u % AHEAD, coming);
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
        coming = rows_of(i + NB + 1 + AHEAD);
      };
      for (int i = 0; i < steps; i += NB) {
        turn(Step<0>{}, i, z[0], z[1]);
        turn(Step<1>{}, i + 1, z[1], z[0]);   // past the last step it finds no keys
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

// ------------------------------------------------------------------ kernels
template <int D, int NW>
__global__ __launch_bounds__(NW * 64, 3) void attend4_rows16_kernel(const AttnArgs a, const Cut c) {
  __shared__ __attribute__((aligned(16))) char smem[Few4<D, NW>::SMEM];
  attend4_rows16<D, NW>(a, c, a.first + (int)blockIdx.x, smem);
}

template <int D, int RG>
__global__ __launch_bounds__(256, 2) void attend4_many_kernel(const AttnArgs a, const Cut c) {
  __shared__ __attribute__((aligned(16))) char smem[Many4<D, RG>::SMEM];
  attend4_many<D, RG>(a, c, a.first + (int)blockIdx.x, smem);
}

// Both kinds of a call in one launch, the tiles of many rows first: the few
// rows' items then fill what those leave of the card.
template <int D, int RG>
__global__ __launch_bounds__(256, 2) void attend4_both_kernel(AttnArgs a, const Join j) {
  constexpr int MANY = Many4<D, RG>::SMEM, FEW = Few4<D, 4>::SMEM;
  __shared__ __attribute__((aligned(16))) char smem[MANY > FEW ? MANY : FEW];
  const int at = j.first + (int)blockIdx.x, k = at < j.items[1];
  a.partial = j.partial[k];
  a.items = j.items[k];
  if (k) attend4_many<D, RG>(a, j.cut[1], at, smem);
  else attend4_rows16<D, 4>(a, j.cut[0], at - j.items[1], smem);
}

template <int D>
hipError_t run(const AttnArgs& a, hipStream_t s) {
  constexpr int NW = 4;
  return run_cuts<D>(
      a, NW * 64, s,
      [&](const AttnArgs& b, const Cut& c, unsigned grid) {
        if (c.R == 16)
          attend4_rows16_kernel<D, NW><<<grid, NW * 64, 0, s>>>(b, c);
        else if (c.R == 64)
          attend4_many_kernel<D, 2><<<grid, 256, 0, s>>>(b, c);
        else
          attend4_many_kernel<D, 4><<<grid, 256, 0, s>>>(b, c);
      },
      [&](const AttnArgs& b, const Join& j, unsigned grid) {
        if (j.cut[1].R == 64) attend4_both_kernel<D, 2><<<grid, 256, 0, s>>>(b, j);
        else attend4_both_kernel<D, 4><<<grid, 256, 0, s>>>(b, j);
      });
}

}  // namespace

hipError_t launch_attention_4bit(const AttnArgs& a, hipStream_t s) {
  return a.dim == 64 ? run<64>(a, s) : run<128>(a, s);
}

}  // namespace bd
