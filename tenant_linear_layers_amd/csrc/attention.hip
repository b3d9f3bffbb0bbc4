// Attention of new tokens over the paged key/value cache.
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
#include <type_traits>

#include "common.h"
#include "e4m3.h"
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

// ------------------------------------------------------------------ few rows
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
    if (only < 0 || ++only > t.i1) return;
    __syncthreads();
  }
}

// Tiles of R rows that the call can have at most.
int64_t most_tiles(const AttnArgs& a, int R) {
  const int64_t all = (int64_t)a.tokens * a.group / R + a.seqs;
  const int64_t by_seq = (int64_t)a.seqs * (((int64_t)a.max_q * a.group + R - 1) / R);
  return all < by_seq ? all : by_seq;
}

// How a call is carried out: sequences of up to 16 rows on the 16-row kernel,
// others on tiles of 64 or 128.  Both kinds in one call are two launches, each
// with a plan of its own sequences.
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

Way way_of(const AttnArgs& a) {
  Way w{};
  const int64_t rows = (int64_t)a.max_q * a.group;
  const int kAll = 2147483647;
  // 128 pieces of little work, not one a CU: their join is longer than what the
  // other CUs would save (a token at 4097 keys 14.2 / 14.8 us, in 8 bits 13.7 /
  // 14.5).  1024 of more: 32 sequences in bf16 152 us, 1280 158 us, 1536 155; 40
  // sequences of 8000 keys 231, 245 and 255 (64 in 8 bits 144, 141 and 141).
  w.cut[0] = Cut{a.group <= 16 ? 16 : 0, 128, 1024, 4, 16, 0, 16, 0.f};
  if (rows > 16) {
    w.cut[1] = Cut{rows_a_tile(a), 512, 512, 8, 64, 0, kAll, 0.f};
    if (a.seqs == 1) w.cut[0].R = 0;   // one sequence: one launch, whatever its length
    if (w.cut[0].R) w.cut[1].least = 16;
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
    if (k == 0 && rows > 16) b.max_q = 16 / a.group;
    w.items[k] = (int)most_items(b, c);
    if (may) w.bytes[k] = (size_t)w.items[k] * c.R * (a.dim + 2) * sizeof(float);
  }
  return w;
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

template <int D, bool Q8>
hipError_t run(AttnArgs a, hipStream_t s) {
  a.by_group = divisor(a.group);
  a.by_page = divisor(a.page);
  a.by_heads = divisor(a.kv_heads);
  const Way w = way_of(a);
  // Waves of a workgroup of few rows: two rings of 64 KB at most fit a CU, and
  // then the second workgroup's start and end lie under the first one's loads.
  // bf16 rows of 128 dims with 2 / 4 waves: a token at 4097 keys 14.2 / 13.9
  // us, 4 of them 22.7 / 27.4, 32 sequences of up to 16000 keys 152 / 156.
  constexpr int NW = !Q8 && D == 128 ? 2 : 4;
  Join j{};
  int joins[2] = {0, 0};
  for (int k = 1; k >= 0; --k) {
    const Cut& c = w.cut[k];
    if (!c.R) continue;
    AttnArgs b = a;
    b.items = w.items[k];
    b.partial = a.partial + (k ? w.bytes[0] / sizeof(float) : 0);
    const int threads = c.R == 16 ? NW * 64 : 256;
    const hipError_t e = in_parts(b.items, threads, [&](int first, unsigned grid) {
      b.first = first;
      if (c.R == 16)
        attend_rows16_kernel<D, Q8, NW, 2><<<grid, NW * 64, 0, s>>>(b, c);
      else if (c.R == 64)
        attend_many_kernel<D, Q8, 2><<<grid, 256, 0, s>>>(b, c);
      else
        attend_many_kernel<D, Q8, 4><<<grid, 256, 0, s>>>(b, c);
    });
    if (e != hipSuccess) return e;
    j.cut[k] = c;
    j.partial[k] = b.partial;
    j.items[k] = b.items;
    if (c.share != 0.f) joins[k] = (b.items - c.target - 8) * (c.R / 16);
  }
  j.from1 = joins[0];
  return in_parts(joins[0] + joins[1], 4 * D, [&](int first, unsigned grid) {
    j.first = first;
    join_pieces_kernel<D><<<grid, 4 * D, 0, s>>>(a, j);
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
  const Way w = way_of(a);
  return w.bytes[0] + w.bytes[1];
}

hipError_t launch_paged_attention(const AttnArgs& a, hipStream_t s) {
  if (a.bits == 4) return launch_attention_4bit(a, s);
  const bool q8 = a.bits == 8;
  if (a.dim == 64) return q8 ? run<64, true>(a, s) : run<64, false>(a, s);
  return q8 ? run<128, true>(a, s) : run<128, false>(a, s);
}

}  // namespace bd
