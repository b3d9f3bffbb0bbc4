// What the attention kernels share: how a call is cut into tiles of rows and
// pieces of their keys, reads of LDS that transpose, and how sums are joined
// and written.
//
// Query i of a sequence with n new tokens and L cached keys (the new ones
// among them) stands at position p = L - n + i and sees the keys j <= p, with
// a window only those with j > p - window:
//
//   o = sum_j exp(z_j - m) v_j / sum_j exp(z_j - m),  z_j = scale q . k_j
//
// One pass over the keys: m is a running reference of the scores and the sums
// (float32) are rescaled when it moves.  The g = heads / kv_heads query heads
// of a key/value head share its keys, so a tile of R rows holds the rows
// r = i g + head of one sequence and key/value head.
//
// Work is cut into items (sequence, tile of rows, piece of the tile's keys,
// key/value head); see Plan.  The pieces of a tile write their sums to the
// workspace and a second kernel joins them.
//
// Operands of the matrix products.  Both are taken transposed, so that a
// query is a column: S^T = K Q^T leaves lane (g4 = lane / 16, n = lane % 16)
// with the scores of query n and the keys 4 g4 .. 4 g4 + 3, and O^T = V^T P^T
// wants from the same lane P of query n at eight keys of its choice, as long
// as V^T has the same keys in the same places.  P therefore goes from one
// product into the other without leaving its lane, and the running maximum
// and sum of a query are held per lane.
#pragma once

#include <type_traits>

#include "common.h"
#include "layer.h"

namespace bd {
namespace {

typedef short s16x4 __attribute__((__vector_size__(8)));
typedef int i32x2 __attribute__((__vector_size__(8)));
#define BD_LDS __attribute__((address_space(3)))

// A tile of up to R rows of one sequence and the keys it can see.
struct Tile {
  int first_q;        // the sequence's first row of q / out
  int row0, rows;     // rows (query * group + head) of the tile
  int pos0;           // position of query 0 of the sequence
  int lo, hi;         // keys that some row of the tile sees
  int all_lo, all_hi; // keys that every row of the tile sees
  int i0, i1;         // its first and last query
};

__device__ __forceinline__ void seq_range(const AttnArgs& a, int b, int& q0, int& n, int& len) {
  q0 = min(max(a.cu_q[b], 0), a.tokens);
  n = max(min(max(a.cu_q[b + 1], 0), a.tokens) - q0, 0);
  len = min(max(a.kv_len[b], 0), a.width * a.page);
}

__device__ __forceinline__ Tile tile_of(const AttnArgs& a, int q0, int n, int len, int t, int R) {
  Tile x;
  x.first_q = q0;
  x.row0 = t * R;
  x.rows = min(R, n * a.group - x.row0);
  x.pos0 = len - n;
  x.i0 = a.by_group.of(x.row0);
  x.i1 = a.by_group.of(x.row0 + x.rows - 1);
  x.hi = max(min(len, x.pos0 + x.i1 + 1), 0);
  x.lo = a.window ? max(x.pos0 + x.i0 - a.window + 1, 0) : 0;
  x.all_hi = x.pos0 + x.i0 + 1;
  x.all_lo = a.window ? x.pos0 + x.i1 - a.window + 1 : 0;
  if (x.lo >= x.hi) x.lo = x.hi = 0;
  return x;
}

// LDS image of key/value rows: the 16-byte pieces of a row are permuted (xor)
// by a function of the row under which 8 rows in a row at one piece (a read of
// K) and 4 rows at a pair of pieces (a transposing read of V) lie in different
// banks: the bits of the row above those that change the bank line, rotated
// left by one.
template <int ROWB>
__device__ __forceinline__ int swizzle(int key) {
  constexpr int P = ROWB / 16, KPL = ROWB >= 256 ? 1 : 256 / ROWB;
  const int x = (key / KPL) & (P - 1);
  return ((x << 1) | (x / (P / 2))) & (P - 1);
}

__device__ __forceinline__ float scale_of(uint32_t dword, int r) {
  return __uint_as_float(((dword >> (8 * r)) & 0xFFu) << 23);
}

// ------------------------------------------------------------------ plan
// The lengths lie on the device, so every workgroup finds its own work: item
// index -> (sequence b, tile, piece of the tile's keys, key/value head), heads
// fastest, pieces next.  A sequence whose widest tile has `blocks` blocks of
// 32 keys is cut into about ceil(blocks / C - 1/2) pieces a tile, with C such
// that all items together are about `round` or `target`; each piece takes an
// equal share of its own tile's blocks.  Then items <= target + tiles *
// kv_heads, which bounds the grid and the workspace on the host.  Every wave
// computes the same plan (lane by sequence, 64 at a time), and the joining
// kernel again.
struct Cut {
  int R;                       // rows a tile
  int round, target;           // items aimed at: of little work, of more
  int min_blocks, enough;      // blocks a piece: at least; for more than one round
  int least, most;             // rows (n * group) of the sequences taken: least < rows <= most
  float share;                 // kv_heads / round; 0: nothing is cut
};

struct Item {
  int b, tile, piece, pieces, head;
  int q0, n, len;
  int first;                   // index of the tile's first piece, by head
};

// One sequence's part of the plan.
struct Seq {
  int q0, n, len, tiles, blocks;
};

__device__ __forceinline__ Seq seq_of(const AttnArgs& a, const Cut& c, int b) {
  Seq s;
  seq_range(a, b, s.q0, s.n, s.len);
  const int rows = s.n * a.group;
  s.tiles = rows > c.least && rows <= c.most ? (rows + c.R - 1) / c.R : 0;  // R: a power of two
  const uint32_t span = (uint32_t)a.window + (uint32_t)min(s.n, c.R);   // keys a tile can see
  const uint32_t keys = a.window ? min((uint32_t)s.len, span) : (uint32_t)s.len;
  s.blocks = (int)((keys + 31) >> 5) + (a.window ? 1 : 0);
  return s;
}

// Item idx (JOIN: tile idx, its first piece); false past the last one.
template <bool JOIN>
__device__ __forceinline__ bool find_item(const AttnArgs& a, const Cut& c, int idx, Item& it) {
  const int lane = threadIdx.x & 63;
  const int want = a.by_heads.of(idx);
  it.head = __builtin_amdgcn_readfirstlane(idx - want * a.kv_heads);
  const bool many = a.seqs > 64;
  Seq s{};
  float load = 0.f;
  int longest = 0;
  for (int b0 = 0; b0 < a.seqs; b0 += 64) {
    float mine = 0.f;
    int blocks = 0;
    if (b0 + lane < a.seqs) {
      s = seq_of(a, c, b0 + lane);
      mine = (float)s.tiles * (float)s.blocks;
      blocks = s.tiles ? s.blocks : 0;
    }
    if (c.share == 0.f) break;
#pragma unroll 1
    for (int o = a.seqs > 1 ? 32 : 0; o > 0; o >>= 1) {
      mine += __shfl_xor(mine, o);
      if (JOIN) blocks = max(blocks, __shfl_xor(blocks, o));
    }
    if (JOIN) longest = max(longest, __builtin_amdgcn_readfirstlane(blocks));
    load += __uint_as_float(__builtin_amdgcn_readfirstlane(__float_as_uint(mine)));
  }
  // `round` pieces for little work, `target` for more: their ends differ by a
  // piece, and a longer piece has its start and end to set against.
  const float few = load * c.share, more = few * ((float)c.round / (float)c.target);
  const float C = fmaxf(floorf(fmaxf(fminf(few, (float)c.enough), more)) + 1.f,
                        (float)c.min_blocks);
  const float per_C = 1.f / C;
  // A rest of half a piece or less is none of its own: 32 sequences in bf16
  // 152 us, with it 163 (64 in 8 bits 144 / 142; 24 mixed ones 30.7 / 30.4).
  auto pieces_of = [&](int blocks) {
    return max((int)fmaf((float)(blocks - 1), per_C, -0.5f) + 1, 1);
  };
  if (JOIN && pieces_of(longest) == 1) return false;   // nothing was cut
  int before = 0, first = 0;   // tiles (JOIN) or items of the chunks before; items of them
  for (int b0 = 0; b0 < a.seqs; b0 += 64) {
    int pieces = 1, items = 0, tl = 0;
    if (b0 + lane < a.seqs) {
      if (many) s = seq_of(a, c, b0 + lane);
      if (c.share != 0.f) pieces = pieces_of(s.blocks);
      items = s.tiles * pieces;
      tl = s.tiles;
    }
    int sum = JOIN ? tl : items, isum = items;
#pragma unroll 1
    for (int o = 1; o < min(a.seqs, 64); o <<= 1) {
      const int up = __shfl_up(sum, o), iup = JOIN ? __shfl_up(isum, o) : 0;
      if (lane >= o) {
        sum += up;
        isum += iup;
      }
    }
    if (!JOIN) isum = sum;
    const int width = JOIN ? tl : items;
    const int at = before + sum - width;
    const uint64_t hit = __ballot(want >= at && want < at + width);
    if (hit) {
      const int src = __builtin_ctzll(hit);
      it.b = b0 + src;
      it.pieces = __builtin_amdgcn_readlane(pieces, src);
      it.q0 = __builtin_amdgcn_readlane(s.q0, src);
      it.n = __builtin_amdgcn_readlane(s.n, src);
      it.len = __builtin_amdgcn_readlane(s.len, src);
      const int local = want - __builtin_amdgcn_readlane(at, src);
      // a sequence's last tiles see the most keys and come first
      const int turn = JOIN || it.pieces == 1 ? local : local / it.pieces;
      it.tile = __builtin_amdgcn_readlane(s.tiles, src) - 1 - turn;
      it.piece = JOIN ? 0 : local - turn * it.pieces;
      it.first = first + __builtin_amdgcn_readlane(isum - items, src) + turn * it.pieces;
      return true;
    }
    const int last = min(a.seqs, 64) - 1;
    before += __builtin_amdgcn_readlane(sum, last);
    first += __builtin_amdgcn_readlane(isum, last);
  }
  return false;
}

// Keys [lo, hi) of a piece: its share of the tile's blocks of 32.
__device__ __forceinline__ void piece_range(const Tile& t, int piece, int pieces, int& lo,
                                            int& hi) {
  lo = t.lo;
  hi = t.hi;
  if (pieces == 1) return;
  const int b0 = t.lo >> 5, nb = t.hi > t.lo ? ((t.hi + 31) >> 5) - b0 : 0;
  const int each = (nb + pieces - 1) / pieces;
  const int from = min(each * piece, nb), to = min(from + each, nb);
  lo = max((b0 + from) << 5, t.lo);
  hi = min((b0 + to) << 5, t.hi);
  if (from == to) lo = hi = 0;
}

// Sums of the pieces: [item][R][D] floats, then [item][R] (m, l).
__device__ __forceinline__ float* sums_at(const AttnArgs& a, const Cut& c, int D, int item) {
  return a.partial + (size_t)item * c.R * D;
}
__device__ __forceinline__ float* ml_at(const AttnArgs& a, const Cut& c, int D, int item) {
  return a.partial + (size_t)a.items * c.R * D + (size_t)item * c.R * 2;
}

// Both launches' pieces: those of cut k in workgroups from[k] on.
struct Join {
  Cut cut[2];
  float* partial[2];
  int items[2], from1;
  int first;   // of this launch's workgroups
};

// A row's sums are held by D / 4 neighbouring lanes, four dims each; a
// workgroup has 16 rows of a tile and head.  Eight pieces are read at once
// (what a call waits for here is the memory's latency, not its rate).  The
// order of the additions is that of the plan, which the lengths alone decide.
template <int D>
__global__ __launch_bounds__(4 * D) void join_pieces_kernel(AttnArgs a, const Join j) {
  const int at = j.first + (int)blockIdx.x, which = at >= j.from1;
  const Cut c = j.cut[which];
  a.partial = j.partial[which];
  a.items = j.items[which];
  const int idx = at - (which ? j.from1 : 0), per = c.R / 16;   // powers of two
  Item it;
  if (!find_item<true>(a, c, idx / per, it) || it.pieces == 1) return;
  // cu_q that does not rise could ask for more items than there are
  if ((it.first + it.pieces) * a.kv_heads > a.items) return;
  const int row = (idx & (per - 1)) * 16 + threadIdx.x / (D / 4);
  const int d0 = threadIdx.x % (D / 4) * 4;
  const int r = it.tile * c.R + row;
  if (r >= it.n * a.group) return;
  const int item0 = it.first * a.kv_heads + it.head;
  float top = -INFINITY, tot = 0.f;
  f32x4 v = {0.f, 0.f, 0.f, 0.f};
  constexpr int U = 8;
#pragma unroll 1
  for (int p0 = 0; p0 < it.pieces; p0 += U) {
    float m[U], l[U];
    f32x4 s[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      m[u] = -INFINITY;
      l[u] = 0.f;
      s[u] = f32x4{0.f, 0.f, 0.f, 0.f};
      if (p0 + u < it.pieces) {
        const int item = item0 + (p0 + u) * a.kv_heads;
        const float* ml = ml_at(a, c, D, item) + row * 2;
        m[u] = ml[0];
        l[u] = ml[1];
        s[u] = *reinterpret_cast<const f32x4*>(sums_at(a, c, D, item) + (size_t)row * D + d0);
      }
    }
    float next = top;
#pragma unroll
    for (int u = 0; u < U; ++u) next = fmaxf(next, m[u]);
    const float ref = next == -INFINITY ? 0.f : next;
    const float old = __builtin_amdgcn_exp2f(top - ref);
    top = next;
    tot *= old;
    v *= old;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const float f = __builtin_amdgcn_exp2f(m[u] - ref);
      tot = fmaf(f, l[u], tot);
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] = fmaf(f, s[u][e], v[e]);
    }
  }
  v *= tot == 0.f ? 0.f : 1.f / tot;
  const int i = a.by_group.of(r);
  uint16_t* o =
      a.out + ((int64_t)(it.q0 + i) * a.heads + it.head * a.group + r - i * a.group) * D + d0;
  *reinterpret_cast<u32x2*>(o) = u32x2{cvt_pk_bf16(v[0], v[1]), cvt_pk_bf16(v[2], v[3])};
}

// ------------------------------------------------------------------ NaN, infinities
// A weight of zero times NaN or infinity is NaN, and the product with V takes
// every key of a step for every row of a tile: a value that is not finite
// would reach rows that do not see it, such as those of the tokens before its
// own.  So a tile whose rows do not all see the same keys looks at its sums
// once they are complete.  Where a row's sums are not finite though its total
// weight is, the item is gone through again for one query at a time, whose
// rows see the same keys; keys outside are read as zeros.
__device__ __forceinline__ bool workgroup_any(bool mine, void* lds) {
  int* found = static_cast<int*>(lds);
  __syncthreads();
  if (threadIdx.x == 0) *found = 0;
  __syncthreads();
  if (mine) *found = 1;
  __syncthreads();
  const int any = *found;
  __syncthreads();
  return any != 0;
}

// Is one of N sums not finite?
template <int N, typename V>
__device__ __forceinline__ bool not_finite(const V* v) {
  float zero = 0.f;
#pragma unroll
  for (int i = 0; i < N; ++i)
#pragma unroll
    for (int r = 0; r < (int)(sizeof(V) / 4); ++r) zero = fmaf(v[i][r], 0.f, zero);
  return zero != 0.f;
}

// The keys of [lo, hi) that query i sees.
__device__ __forceinline__ void query_range(const AttnArgs& a, const Tile& t, int i, int& lo,
                                            int& hi) {
  hi = min(hi, t.pos0 + i + 1);
  if (a.window) lo = max(lo, t.pos0 + i - a.window + 1);
  if (lo >= hi) lo = hi = 0;
}

// ------------------------------------------------------------------ weights
// Two weights as the product with V takes them, and their part of the total.
// They are rounded to bf16: the matrix cores take both operands in one type,
// and bf16 is that of V.  The total is that of the rounded weights, in float32:
// what is left of the rounding is the mean of 2^-9 (v_j - o) over the keys, so
// rows of one value give that value (over 16 keys whose heaviest stands 2^5.3
// above the reference an error of 0.0013 of the output, 0.0025 against the total
// before rounding; over 16000 keys 0.0020 and 0.0021).  A second product with
// what the rounding leaves off would take that error away: for few rows it costs
// 0 to 3.5% (a token at 4097 keys 14.3 / 14.8 us, 40 sequences of 8000 233 / 237),
// for many it is half as many matrix products again.
__device__ __forceinline__ uint32_t weights(float p0, float p1, float& l) {
  const uint32_t two = cvt_pk_bf16(p0, p1);
  l = __builtin_amdgcn_fdot2_f32_bf16(__builtin_bit_cast(bf16x2, two),
                                      __builtin_bit_cast(bf16x2, 0x3F803F80u), l, false);
  return two;
}

// ------------------------------------------------------------------ reads of V
// Transposing LDS reads: 16 lanes read 8 bytes each, together a block of four
// rows of 16 bf16 (eight rows of 16 bytes), and lane n of them gets column n.
__device__ __forceinline__ u32x2 read_tr16(char* p) {
  return __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((BD_LDS s16x4*)p));
}

// Several at once, their wait in the same statement: under the 16-row kernel's
// ring the builtin would also wait for every load to LDS in flight, the next
// steps' among them.
__device__ __forceinline__ uint32_t lds_address(const void* p) {
  return (uint32_t)(uintptr_t)(BD_LDS const char*)p;
}

// Blocks of four rows at four addresses and OFF bytes after each.
template <int OFF>
__device__ __forceinline__ void read_tr16(const uint32_t (&at)[4], u32x4 (&v)[4]) {
  u32x2 r[8];
  asm volatile(
      "ds_read_b64_tr_b16 %0, %8\n"
      "ds_read_b64_tr_b16 %1, %8 offset:%12\n"
      "ds_read_b64_tr_b16 %2, %9\n"
      "ds_read_b64_tr_b16 %3, %9 offset:%12\n"
      "ds_read_b64_tr_b16 %4, %10\n"
      "ds_read_b64_tr_b16 %5, %10 offset:%12\n"
      "ds_read_b64_tr_b16 %6, %11\n"
      "ds_read_b64_tr_b16 %7, %11 offset:%12\n"
      "s_waitcnt lgkmcnt(0)"
      : "=&v"(r[0]), "=&v"(r[1]), "=&v"(r[2]), "=&v"(r[3]), "=&v"(r[4]), "=&v"(r[5]),
        "=&v"(r[6]), "=&v"(r[7])
      : "v"(at[0]), "v"(at[1]), "v"(at[2]), "v"(at[3]), "n"(OFF)
      : "memory");
#pragma unroll
  for (int i = 0; i < 4; ++i)
    v[i] = u32x4{r[2 * i][0], r[2 * i][1], r[2 * i + 1][0], r[2 * i + 1][1]};
}

__device__ __forceinline__ void read_tr8(const uint32_t (&at)[4], u32x2 (&r)[4]) {
  asm volatile(
      "ds_read_b64_tr_b8 %0, %4\n"
      "ds_read_b64_tr_b8 %1, %5\n"
      "ds_read_b64_tr_b8 %2, %6\n"
      "ds_read_b64_tr_b8 %3, %7\n"
      "s_waitcnt lgkmcnt(0)"
      : "=&v"(r[0]), "=&v"(r[1]), "=&v"(r[2]), "=&v"(r[3])
      : "v"(at[0]), "v"(at[1]), "v"(at[2]), "v"(at[3])
      : "memory");
}

// ------------------------------------------------------------------ waits
template <int N>
__device__ __forceinline__ void wait_loads() {   // at most N vector loads in flight
  __builtin_amdgcn_sched_barrier(0);
  __builtin_amdgcn_s_waitcnt((N & 15) | ((N >> 4) << 14) | (0x7 << 4) | (0xF << 8));
  __builtin_amdgcn_sched_barrier(0);
}
__device__ __forceinline__ void wait_lds() {
  __builtin_amdgcn_s_waitcnt(0xC07F);  // lgkmcnt(0)
  __builtin_amdgcn_sched_barrier(0);
}

// ------------------------------------------------------------------ results
// The sums of a workgroup of the 16-row kernel, one set a wave: lane (n, g4)
// has row n and the dims 16 d + 4 g4 .. + 3 of acc[d].  only: the query that
// is written, or -1 for all.
template <int D, int NW>
__device__ __forceinline__ void write_rows16(const AttnArgs& a, const Cut& c, const Item& it,
                                             const Tile& t, char* smem, int wv, int n, int g4,
                                             const f32x4 (&acc)[D / 16], float m, float l,
                                             int only) {
  constexpr int R = 16;
  // Join of the waves: [wave][row] m, l, then [wave][row][D] sums.
  __syncthreads();
  float* ml = reinterpret_cast<float*>(smem);
  float* sums = ml + NW * R * 2;
  if (g4 == 0) {
    ml[(wv * R + n) * 2] = m;
    ml[(wv * R + n) * 2 + 1] = l;
  }
#pragma unroll
  for (int dt = 0; dt < D / 16; ++dt)
    *reinterpret_cast<f32x4*>(sums + (wv * R + n) * D + dt * 16 + 4 * g4) = acc[dt];
  __syncthreads();
  constexpr int TPR = NW * 64 / R;          // threads a row
  const int row = threadIdx.x / TPR;
  const int i = a.by_group.of(t.row0 + row);
  if (row < t.rows && (only < 0 || i == only)) {
    float top = -INFINITY;
#pragma unroll
    for (int w = 0; w < NW; ++w) top = fmaxf(top, ml[(w * R + row) * 2]);
    const float ref = top == -INFINITY ? 0.f : top;
    float f[NW], tot = 0.f;
#pragma unroll
    for (int w = 0; w < NW; ++w) {
      f[w] = __builtin_amdgcn_exp2f(ml[(w * R + row) * 2] - ref);
      tot += f[w] * ml[(w * R + row) * 2 + 1];
    }
    const bool whole = it.pieces == 1;
    // a row that sees nothing: zeros
    const float inv = !whole ? 1.f : tot == 0.f ? 0.f : 1.f / tot;
    uint16_t* o = a.out + ((int64_t)(t.first_q + i) * a.heads + it.head * a.group +
                           (t.row0 + row) - i * a.group) * D;
    const int item = (it.first + it.piece) * a.kv_heads + it.head;
    if (!whole && threadIdx.x % TPR == 0) {
      float* p = ml_at(a, c, D, item) + row * 2;
      p[0] = top;
      p[1] = tot;
    }
#pragma unroll
    for (int k = 0; k < D / (4 * TPR); ++k) {
      const int d0 = (k * TPR + threadIdx.x % TPR) * 4;
      f32x4 v = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int w = 0; w < NW; ++w)
        v += f[w] * *reinterpret_cast<const f32x4*>(sums + (w * R + row) * D + d0);
      v *= inv;
      if (whole)
        *reinterpret_cast<u32x2*>(o + d0) =
            u32x2{cvt_pk_bf16(v[0], v[1]), cvt_pk_bf16(v[2], v[3])};
      else
        *reinterpret_cast<f32x4*>(sums_at(a, c, D, item) + row * D + d0) = v;
    }
  }
}

// Those of tiles of 32 RG rows: a wave has the 32 rows rg of key group kg, lane
// (n, hh) row n and the dims 32 d + 8 r + 4 hh .. + 3 in acc[d][4 r] and on.
template <int D, int RG>
__device__ __forceinline__ void write_many(const AttnArgs& a, const Cut& c, const Item& it,
                                           const Tile& t, char* smem, int rg, int kg, int n,
                                           int hh, int my, int qi, const f32x16 (&acc)[D / 32],
                                           float m, float l, int only) {
  constexpr int KG = 4 / RG, R = 32 * RG;
  const bool whole = it.pieces == 1;
  const int item = (it.first + it.piece) * a.kv_heads + it.head;
  if (KG == 1) {
    const int row = 32 * rg + n;
    if (row < t.rows && (only < 0 || qi == only)) {
      uint16_t* o = a.out + ((int64_t)(t.first_q + qi) * a.heads + it.head * a.group + my -
                             qi * a.group) * D;
      const float inv = l == 0.f ? 0.f : 1.f / l;   // a row that sees nothing: zeros
      if (!whole && hh == 0) {
        float* p = ml_at(a, c, D, item) + row * 2;
        p[0] = m;
        p[1] = l;
      }
#pragma unroll
      for (int d = 0; d < D / 32; ++d)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const f32x4 v = {acc[d][4 * r], acc[d][4 * r + 1], acc[d][4 * r + 2],
                           acc[d][4 * r + 3]};
          const int d0 = 32 * d + 8 * r + 4 * hh;
          if (whole)
            *reinterpret_cast<u32x2*>(o + d0) =
                u32x2{cvt_pk_bf16(v[0] * inv, v[1] * inv), cvt_pk_bf16(v[2] * inv, v[3] * inv)};
          else
            *reinterpret_cast<f32x4*>(sums_at(a, c, D, item) + (size_t)row * D + d0) = v;
        }
    }
  } else {
    // Join of the groups: [group][row] m, l, then [group][row][D] sums.
    __syncthreads();
    float* ml = reinterpret_cast<float*>(smem);
    float* sums = ml + KG * R * 2;
    const int at = kg * R + 32 * rg + n;
    if (hh == 0) {
      ml[at * 2] = m;
      ml[at * 2 + 1] = l;
    }
#pragma unroll
    for (int d = 0; d < D / 32; ++d)
#pragma unroll
      for (int r = 0; r < 4; ++r)
        *reinterpret_cast<f32x4*>(sums + at * D + 32 * d + 8 * r + 4 * hh) =
            f32x4{acc[d][4 * r], acc[d][4 * r + 1], acc[d][4 * r + 2], acc[d][4 * r + 3]};
    __syncthreads();
    constexpr int TPR = D / 4, RPP = 256 / TPR;   // threads a row, rows a pass
    for (int row = threadIdx.x / TPR; row < t.rows; row += RPP) {
      const int i = a.by_group.of(t.row0 + row);
      if (only >= 0 && i != only) continue;
      float top = -INFINITY;
#pragma unroll
      for (int w = 0; w < KG; ++w) top = fmaxf(top, ml[(w * R + row) * 2]);
      const float ref = top == -INFINITY ? 0.f : top;
      const int d0 = (threadIdx.x % TPR) * 4;
      float tot = 0.f;
      f32x4 v = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int w = 0; w < KG; ++w) {
        const float f = __builtin_amdgcn_exp2f(ml[(w * R + row) * 2] - ref);
        tot += f * ml[(w * R + row) * 2 + 1];
        v += f * *reinterpret_cast<const f32x4*>(sums + (w * R + row) * D + d0);
      }
      if (whole) {
        v *= tot == 0.f ? 0.f : 1.f / tot;
        uint16_t* o = a.out + ((int64_t)(t.first_q + i) * a.heads + it.head * a.group +
                               (t.row0 + row) - i * a.group) * D;
        *reinterpret_cast<u32x2*>(o + d0) =
            u32x2{cvt_pk_bf16(v[0], v[1]), cvt_pk_bf16(v[2], v[3])};
      } else {
        *reinterpret_cast<f32x4*>(sums_at(a, c, D, item) + (size_t)row * D + d0) = v;
        if (d0 == 0) {
          float* p = ml_at(a, c, D, item) + row * 2;
          p[0] = top;
          p[1] = tot;
        }
      }
    }
  }
}

// ------------------------------------------------------------------ on the host
// Tiles of R rows that the call can have at most.
int64_t most_tiles(const AttnArgs& a, int R) {
  const int64_t all = (int64_t)a.tokens * a.group / R + a.seqs;
  const int64_t by_seq = (int64_t)a.seqs * (((int64_t)a.max_q * a.group + R - 1) / R);
  return all < by_seq ? all : by_seq;
}

// How a call is carried out: sequences of few rows on the 16-row kernel,
// others on tiles of 64 or 128.  Both kinds in one call have each a plan of its own
// sequences, in two launches or, over 4 bits, in one.
struct Way {
  Cut cut[2];        // few rows, many rows; R = 0: no such sequences
  int items[2];      // grids
  size_t bytes[2];   // workspaces
};

// Items that the plan can have at most.
int64_t most_items(const AttnArgs& a, const Cut& c) {
  return most_tiles(a, c.R) * a.kv_heads + (c.share != 0.f ? c.target + 8 : 0);
}

// Rows of a tile of many rows.  128 rows read half of what tiles of 64 read
// and need not share a workgroup's keys out: 200 tokens over 8000 keys, 4 rows
// a token, 54 us against 77 (8 bits, 128 dims; of 64 dims 41 against 53).  64
// where
// * the average sequence would leave 128 too empty (40 tokens, 160 rows, over
//   8000 keys: 30.5 us against 33.0; of 64 dims 24.9 against 29.1), or
// * the tiles of 128 are about one round of the card, 512, and their lengths
//   differ, new tokens being about half or more of the keys: a long tile is then
//   what the call waits for.  The more tiles there are, the longer the sequences
//   have to be for that, and half as much again for 64 dims, whose steps are
//   shorter against what a workgroup starts and ends with (us with tiles of 64 /
//   of 128; 8 bits in brackets):
//     280 tokens of 64 heads, 136 tiles   21.8 / 21.4   (fewer than 200: 24.0 / 22.4)
//     512 of 64 heads, 256 tiles          20.6 / 32.5   (22.9 / 34.3)
//     800 of 64 heads, 400                36.8 / 36.3   (40.6 / 39.1)
//     1200 of 64 heads, 600               59.6 / 42.7   (65.6 / 44.4)
//     1200 of 32 heads, 296               30.8 / 42.8   (35.1 / 44.8)
//     1600 of 32 heads, 400               47.0 / 53.5   (51.5 / 56.7)
//     2400 of 32 heads, 600               83.1 / 71.5   (91.6 / 75.6)
//     4800 of 16 heads, 600               131.2 / 129.0 (144.4 / 136.3)
//     4 sequences of 200, 64 heads, 400   37.1 / 25.1   (40.9 / 26.4)
//     64 dims: 800 of 64 heads, 400       21.0 / 26.0   (27.3 / 29.7)
//              1200 of 64 heads, 600      34.2 / 29.6   (42.8 / 33.5)
//              2048 of 32 heads, 512      39.4 / 42.5   (45.6 / 48.5)
//              4800 of 16 heads, 600      80.7 / 89.7   (92.8 / 101.4)
//   Over 1.25 times as many cached keys 64 rows are slower where sequences are
//   long (1680 tokens of 16 heads 69 / 69, in 8 bits 77 / 73; of 32 heads 125 /
//   111), not where they are short (420 of 64 heads 31 / 38).
int rows_a_tile(const AttnArgs& a) {
  const int64_t all = (int64_t)a.tokens * a.group, each = all / a.seqs;
  const bool filled = (each + 127) / 128 * 128 * 4 <= (each + 63) / 64 * 64 * 5;
  const int64_t tiles = all / 128 * a.kv_heads;
  const int64_t most = 200 + a.max_q / (a.dim == 64 ? 4 : 6);
  const bool uneven = tiles >= 200 && tiles < (most < 1000 ? most : 1000) &&
                      (int64_t)a.max_q * 9 >= (int64_t)a.width * a.page * 4;
  return filled && !uneven ? 128 : 64;
}

Way way_with(const AttnArgs& a, int few) {   // sequences of up to `few` rows by 16
  Way w{};
  const int64_t rows = (int64_t)a.max_q * a.group;
  const int kAll = 2147483647;
  // 128 pieces of little work, not one a CU: their join is longer than what the
  // other CUs would save (a token at 4097 keys 14.2 / 14.8 us, in 8 bits 13.7 /
  // 14.5).  1024 of more: 32 sequences in bf16 152 us, 1280 158 us, 1536 155; 40
  // sequences of 8000 keys 231, 245 and 255 (64 in 8 bits 144, 141 and 141).  768
  // over 4 bits of 128 dims, the three workgroups of a CU (with 1024 / 768: 32
  // sequences of 8000 keys 60.6 / 57.3, 10 of 16000 46.5 / 43.1, 24 of up to 16000
  // 47.2 / 45.3, 64 88 / 88, 16 tokens over 8000 25.5 / 22.1; but where that leaves
  // a short second round 20 sequences of 12000 56.9 / 62.2, 40 of 8000 69.6 / 72.5).
  const int target = a.bits == 4 && a.dim == 128 ? 768 : 1024;
  w.cut[0] = Cut{a.group <= few ? 16 : 0, 128, target, 4, 16, 0, few, 0.f};
  if (rows > few) {
    w.cut[1] = Cut{rows_a_tile(a), 512, 512, 8, 64, 0, kAll, 0.f};
    if (a.seqs == 1) w.cut[0].R = 0;   // one sequence: one launch, whatever its length
    if (w.cut[0].R) {
      w.cut[1].least = few;
      // The kernel of both kinds has the registers of its tiles of many rows: over 4
      // bits two workgroups of 128 dims a CU, three of 64.  60 single tokens and 4 of
      // 20 over 4000 keys with 768 / 512 98.5 / 92 us, 60 and one of 20 80.5 / 74, 200
      // tokens over 4000 with 40 single ones over 8000 124 / 126; of 64 dims, with 1024
      // / 768, 200 with 40 75 / 72, 24 mixed ones 37.2 / 36.4, others alike.
      if (a.bits == 4) w.cut[0].target = a.dim == 128 ? 512 : 768;
    }
  }
  for (int k = 0; k < 2; ++k) {
    Cut& c = w.cut[k];
    if (!c.R) continue;
    // Cut only where a tile can be longer than the shortest piece, and, for many
    // rows, where the tiles by themselves are not a round of the card, 512: a cut
    // call has its join (5 us and more) and its pieces' sums to set against
    // shorter ends.  64 heads, whole / cut: 1060 tokens, 528 tiles, 38.1 / 46.4
    // us, 1060 over 4240 cached 251 / 259, 2000 tokens 83 / 97, 2048 86 / 100; 420
    // over 1680, 208 tiles, 55 / 55, over 6720 175 / 134.  (From nothing whole
    // tiles are faster below a round too: 840 tokens, 416 tiles, 32 / 39.)
    // Sequences whose cached keys may be many times their new ones can be of very
    // different lengths, and are cut up to two rounds: 8 sequences of 128 tokens
    // over 0 to 12000 keys, 512 tiles, 207 / 113; of 128 tokens and no more 24 / 25,
    // of 300 to 600 tokens, 880 tiles, 50 / 64.
    // Pieces of 8 blocks or more: of 16, 16 tokens of 64 heads over 1500 keys take
    // 23 us for 19, over 8000 29 for 31, 512 from nothing, of 32 heads, 21 for 24.
    const int64_t keys = (int64_t)a.width * a.page;
    const bool alike = a.seqs == 1 || keys <= 4 * (int64_t)a.max_q;
    const bool may = (keys + 31) / 32 + 1 > c.min_blocks &&
                     (k == 0 || (int64_t)a.tokens * a.group / c.R * a.kv_heads <
                                    (alike ? c.target : 2 * c.target));
    c.share = may ? (float)a.kv_heads / (float)c.round : 0.f;
    AttnArgs b = a;
    if (k == 0 && rows > few) b.max_q = few / a.group;
    w.items[k] = (int)most_items(b, c);
    if (may) w.bytes[k] = (size_t)w.items[k] * c.R * (a.dim + 2) * sizeof(float);
  }
  return w;
}

// Bytes of a plan's sums.
size_t way_bytes(const Way& w) { return w.bytes[0] + w.bytes[1]; }

// The plan of bf16 and e4m3 caches, and what the workspace is sized by for every
// type: a caller asks for the size without naming one.
Way way_of_size(AttnArgs a) {
  a.bits = 16;
  return way_with(a, 16);
}

// Over 4 bits, where keys are cheap to read again, sequences of up to 32 rows go
// by 16 too (us so / on tiles of 64 or 128 rows; 8 key/value heads of 128 dims: 4
// new tokens of 64 heads over 8000 keys 14.6 / 28.9, 16 such sequences over 4000
// 31.4 / 42.6, 64 over 1000 32.6 / 44.6), and all of a call whose tiles of 16 are
// less than a workgroup a CU (8 tokens over 8000 17.6 / 31.4, 16 22.1 / 33.2, 4
// sequences of 8, 128 tiles, 29.9 / 36.2, 1000 from nothing of 2 heads 13.0 / 18.7;
// but 4 of 16, 256 tiles, 43.5 / 40.1, 8 of 8 44.0 / 42.9, of 64 dims 29.7 / 28.5).
// Beside longer ones too: 20 single tokens, 20 of 4 and one of 100 over 4000 keys 86 /
// 97, 32 of 3 with one of 64 over 2000 52 / 61, 16 of 4 with one of 200 over 4000 83 /
// 87.5, of 64 dims 49 / 62.
// A plan is taken only where it fits into the workspace that way_of_size asks for
// (with very many sequences, such as 100 of 4 tokens with one of 100, the one by 32
// does not); way_of_size itself is the last, so no target above has to be below another.
Way way_of(const AttnArgs& a) {
  const Way all = way_of_size(a);
  if (a.bits != 4) return all;
  for (int few : {most_tiles(a, 16) * a.kv_heads <= 192 ? 2147483647 : 32, 16}) {
    const Way w = way_with(a, few);
    if (way_bytes(w) <= way_bytes(all)) return w;
  }
  return all;
}

// A launch takes fewer than 2^32 threads: more workgroups than that go in
// several, of 2^31 threads each.
template <typename F>
hipError_t in_parts(int grid, int threads, F launch) {
  const int most = (int)((int64_t(1) << 31) / threads);
  for (int at = 0; at < grid; at += most) {
    launch(at, (unsigned)(grid - at < most ? grid - at : most));
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

// A call: the launches of its cuts, then the join of what they cut.
// start(b, c, grid) starts `grid` workgroups of cut c, of few_threads threads
// (R = 16) or 256.  both(b, j, grid), where there is one, starts those of both
// cuts, of 256 threads, cut 1's first.
struct Apart {};   // no `both`
template <int D, typename F, typename G = Apart>
hipError_t run_cuts(AttnArgs a, int few_threads, hipStream_t s, F start, G both = G{}) {
  a.by_group = divisor(a.group);
  a.by_page = divisor(a.page);
  a.by_heads = divisor(a.kv_heads);
  const Way w = way_of(a);
  Join j{};
  int joins[2] = {0, 0};
  for (int k = 0; k < 2; ++k) {
    const Cut& c = w.cut[k];
    if (!c.R) continue;
    j.cut[k] = c;
    j.partial[k] = a.partial + (k ? w.bytes[0] / sizeof(float) : 0);
    j.items[k] = w.items[k];
    if (c.share != 0.f) joins[k] = (w.items[k] - c.target - 8) * (c.R / 16);
  }
  hipError_t e = hipSuccess;
  bool apart = true;
  if constexpr (!std::is_same_v<G, Apart>) {
    const int64_t all = (int64_t)j.items[0] + j.items[1];
    if (j.items[0] && j.items[1] && all <= 2147483647) {
      apart = false;
      e = in_parts((int)all, 256, [&](int first, unsigned grid) {
        j.first = first;
        both(a, j, grid);
      });
    }
  }
  for (int k = 1; apart && k >= 0 && e == hipSuccess; --k) {
    AttnArgs b = a;
    b.items = j.items[k];
    b.partial = j.partial[k];
    e = in_parts(b.items, j.cut[k].R == 16 ? few_threads : 256, [&](int first, unsigned grid) {
      b.first = first;
      start(b, j.cut[k], grid);
    });
  }
  if (e != hipSuccess) return e;
  j.from1 = joins[0];
  return in_parts(joins[0] + joins[1], 4 * D, [&](int first, unsigned grid) {
    j.first = first;
    join_pieces_kernel<D><<<grid, 4 * D, 0, s>>>(a, j);
  });
}

}  // namespace
}  // namespace bd
