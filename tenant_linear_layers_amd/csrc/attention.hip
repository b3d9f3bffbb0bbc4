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
#include "common.h"
#include "e4m3.h"
#include "layer.h"

namespace bd {
namespace {

typedef uint32_t u32x2 __attribute__((__vector_size__(8)));
typedef u32x4 u32x4_any __attribute__((aligned(2)));  // strided rows of any alignment
typedef short s16x4 __attribute__((__vector_size__(8)));
typedef int i32x2 __attribute__((__vector_size__(8)));
#define BD_LDS __attribute__((address_space(3)))

// A tile of up to R rows of one sequence and the keys it can see.
struct Tile {
  int first_q, n_q;   // the sequence's rows of q / out and their number
  int row0, rows;     // rows (query * group + head) of the tile
  int pos0;           // position of query 0 of the sequence
  int lo, hi;         // keys that some row of the tile sees
};

__device__ __forceinline__ void seq_range(const AttnArgs& a, int b, int& q0, int& n, int& len) {
  q0 = min(max(a.cu_q[b], 0), a.tokens);
  n = max(min(max(a.cu_q[b + 1], 0), a.tokens) - q0, 0);
  len = min(max(a.kv_len[b], 0), a.width * a.page);
}

__device__ __forceinline__ Tile tile_of(const AttnArgs& a, int q0, int n, int len, int t, int R) {
  Tile x;
  x.first_q = q0;
  x.n_q = n;
  x.row0 = t * R;
  x.rows = min(R, n * a.group - x.row0);
  x.pos0 = len - n;
  const int i0 = x.row0 / a.group, i1 = (x.row0 + x.rows - 1) / a.group;
  x.hi = max(min(len, x.pos0 + i1 + 1), 0);
  x.lo = a.window ? max(x.pos0 + i0 - a.window + 1, 0) : 0;
  if (x.lo >= x.hi) x.lo = x.hi = 0;
  return x;
}

// LDS image of key/value rows: 16-byte pieces of a row permuted by the row
// so that both readers below meet all the banks.
template <int ROWB>
__device__ __forceinline__ int swizzle(int key) {
  constexpr int P = ROWB / 16, KPL = ROWB >= 256 ? 1 : 256 / ROWB;
  return (key / KPL) & (P - 1);
}

__device__ __forceinline__ float scale_of(uint32_t dword, int r) {
  return __uint_as_float(((dword >> (8 * r)) & 0xFFu) << 23);
}

// ------------------------------------------------------------------ few rows
// Tiles of 16 rows.  The four waves of a workgroup take 32-key steps of the
// tile's keys in turn, each through its own part of LDS, and join at the end.
template <int D, bool Q8>
__global__ __launch_bounds__(256) void attend_rows16_kernel(const AttnArgs a) {
  constexpr int R = 16, NW = 4;
  constexpr int ROWB = Q8 ? D : 2 * D;
  constexpr int P = ROWB / 16;              // 16-byte pieces of a row
  constexpr int KPI = 64 / P;               // keys per staging instruction
  constexpr int STAGE = 32 * ROWB;          // one of K, V
  constexpr int RED = NW * R * (D + 2) * 4;
  constexpr int SMEM = NW * 2 * STAGE > RED ? NW * 2 * STAGE : RED;
  __shared__ __attribute__((aligned(16))) char smem[SMEM];

  const int lane = threadIdx.x & 63;
  const int wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int n = lane & 15, g4 = lane >> 4;
  const int head = blockIdx.x;   // key/value head
  const int b = blockIdx.z;
  int q0, nq, len;
  seq_range(a, b, q0, nq, len);
  if ((int)blockIdx.y * R >= nq * a.group) return;
  const Tile t = tile_of(a, q0, nq, len, blockIdx.y, R);

  // Q^T: lane n's row, the dims that the lane's K pieces hold.
  u32x4 qf[D / 32];
  const int my = min(n, t.rows - 1);
  const int qi = (t.row0 + my) / a.group;
  const uint16_t* qp = a.q + (int64_t)(t.first_q + qi) * a.q_token_stride +
                       (int64_t)(head * a.group + (t.row0 + my) - qi * a.group) * a.q_head_stride;
#pragma unroll
  for (int s = 0; s < D / 32; ++s) {
    const int d0 = Q8 ? 64 * (s >> 1) + 16 * g4 + 8 * (s & 1) : 32 * s + 8 * g4;
    qf[s] = *reinterpret_cast<const u32x4_any*>(qp + d0);
  }
  const int pos = t.pos0 + qi;
  const int vis_hi = pos + 1, vis_lo = a.window ? pos - a.window + 1 : 0;

  char* kst = smem + wv * 2 * STAGE;
  char* vst = kst + STAGE;
  f32x4 acc[D / 16];
#pragma unroll
  for (int i = 0; i < D / 16; ++i) acc[i] = f32x4{0.f, 0.f, 0.f, 0.f};
  float m = -INFINITY, l = 0.f;
  bool bad = false;

  for (int key0 = (t.lo & ~31) + 32 * wv; key0 < t.hi; key0 += 32 * NW) {
    uint32_t ks[2] = {0, 0}, vs[2] = {0, 0};
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int k0 = key0 + 16 * h;
      int page = 0;
      if (k0 < t.hi) {
        page = a.table[(int64_t)b * a.width + k0 / a.page];
        if (page < 0 || page >= a.pages) bad = true;
      }
      const int keys = page < 0 || page >= a.pages ? 0 : min(max(t.hi - k0, 0), 16);
      const int64_t row = ((int64_t)(keys ? page : 0) * a.kv_heads + head) * a.page + k0 % a.page;
#pragma unroll
      for (int j = 0; j < 16 / KPI; ++j) {
        const int key = j * KPI + lane / P, piece = lane % P;
        u32x4 kv = {0, 0, 0, 0}, vv = {0, 0, 0, 0};
        if (key < keys && k0 + key >= t.lo) {
          kv = ld128(a.cache[0] + (row + key) * ROWB + piece * 16);
          vv = ld128(a.cache[1] + (row + key) * ROWB + piece * 16);
        }
        const int at = (16 * h + key) * ROWB + ((piece ^ swizzle<ROWB>(16 * h + key)) << 4);
        *reinterpret_cast<u32x4*>(kst + at) = kv;
        *reinterpret_cast<u32x4*>(vst + at) = vv;
      }
      if (Q8 && keys) {
        ks[h] = ld32(a.scale[0] + row + 4 * g4);
        vs[h] = ld32(a.scale[1] + row + 4 * g4);
      }
    }
    __builtin_amdgcn_s_waitcnt(0xC07F);  // lgkmcnt(0): the wave's own stage is written
    __builtin_amdgcn_sched_barrier(0);

    float s[8];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      f32x4 z = {0.f, 0.f, 0.f, 0.f};
      const int key = 16 * h + n;
      if (Q8) {
#pragma unroll
        for (int p = 0; p < D / 64; ++p) {
          const u32x4 c = *reinterpret_cast<const u32x4*>(
              kst + key * ROWB + (((4 * p + g4) ^ swizzle<ROWB>(key)) << 4));
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const u32x4 kf = {bf16x2_of_e4m3<false>(c[2 * e], 1.f),
                              bf16x2_of_e4m3<true>(c[2 * e], 1.f),
                              bf16x2_of_e4m3<false>(c[2 * e + 1], 1.f),
                              bf16x2_of_e4m3<true>(c[2 * e + 1], 1.f)};
            z = mfma16(kf, qf[2 * p + e], z);
          }
        }
      } else {
#pragma unroll
        for (int p = 0; p < D / 32; ++p)
          z = mfma16(*reinterpret_cast<const u32x4*>(
                         kst + key * ROWB + (((4 * p + g4) ^ swizzle<ROWB>(key)) << 4)),
                     qf[p], z);
      }
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int j = key0 + 16 * h + 4 * g4 + r;
        float v = z[r] * a.scale_log2;
        if (Q8) v *= scale_of(ks[h], r);
        s[4 * h + r] = j < vis_hi && j >= vis_lo && j < t.hi ? v : -INFINITY;
      }
    }
    float top = s[0];
#pragma unroll
    for (int e = 1; e < 8; ++e) top = fmaxf(top, s[e]);
    top = fmaxf(top, __shfl_xor(top, 16));
    top = fmaxf(top, __shfl_xor(top, 32));
    const float m1 = fmaxf(m, top);
    const float ref = m1 == -INFINITY ? 0.f : m1;
    const float f = __builtin_amdgcn_exp2f(m - ref);
    m = m1;
    l *= f;
#pragma unroll
    for (int i = 0; i < D / 16; ++i) acc[i] *= f;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      s[e] = __builtin_amdgcn_exp2f(s[e] - ref);
      l += s[e];
      if (Q8) s[e] = s[e] > 0.f ? s[e] * scale_of(vs[e >> 2], e & 3) : 0.f;  // 0 past the end
    }
    const u32x4 pf = {cvt_pk_bf16(s[0], s[1]), cvt_pk_bf16(s[2], s[3]), cvt_pk_bf16(s[4], s[5]),
                      cvt_pk_bf16(s[6], s[7])};
#pragma unroll
    for (int dt = 0; dt < D / 16; ++dt) {
      u32x4 vf;
      if (Q8) {
        // eight keys (4 g4 + 0..3 of both halves) of one dim per lane
        const int key = 16 * (n >> 3) + 4 * g4 + ((n >> 1) & 3);
        const i32x2 c = __builtin_amdgcn_ds_read_tr8_b64_v2i32(
            (BD_LDS i32x2*)(vst + key * ROWB + ((dt ^ swizzle<ROWB>(key)) << 4) + 8 * (n & 1)));
        vf = u32x4{bf16x2_of_e4m3<false>(c[0], 1.f), bf16x2_of_e4m3<true>(c[0], 1.f),
                   bf16x2_of_e4m3<false>(c[1], 1.f), bf16x2_of_e4m3<true>(c[1], 1.f)};
      } else {
        u32x2 c[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int key = 16 * h + 4 * g4 + (n >> 2);
          c[h] = __builtin_bit_cast(
              u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((BD_LDS s16x4*)(
                         vst + key * ROWB +
                         (((2 * dt + ((n >> 1) & 1)) ^ swizzle<ROWB>(key)) << 4) + 8 * (n & 1))));
        }
        vf = u32x4{c[0][0], c[0][1], c[1][0], c[1][1]};
      }
      acc[dt] = mfma16(vf, pf, acc[dt]);
    }
    __builtin_amdgcn_s_waitcnt(0xC07F);  // the stage has been read before it is written again
    __builtin_amdgcn_sched_barrier(0);
  }
  if (bad) l = NAN;
  l += __shfl_xor(l, 16);
  l += __shfl_xor(l, 32);

  // Join of the four waves: [wave][row] m, l, then [wave][row][D] sums.
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
  const int row = threadIdx.x >> 4;
  if (row >= t.rows) return;
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
  const float inv = tot == 0.f ? 0.f : 1.f / tot;  // a row that sees nothing gives zeros
  const int i = (t.row0 + row) / a.group;
  uint16_t* o = a.out + ((int64_t)(t.first_q + i) * a.heads + head * a.group + (t.row0 + row) -
                         i * a.group) * D;
#pragma unroll
  for (int c = 0; c < D / 64; ++c) {
    const int d0 = c * 64 + (threadIdx.x & 15) * 4;
    f32x4 v = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int w = 0; w < NW; ++w)
      v += f[w] * *reinterpret_cast<const f32x4*>(sums + (w * R + row) * D + d0);
    v *= inv;
    *reinterpret_cast<u32x2*>(o + d0) = u32x2{cvt_pk_bf16(v[0], v[1]), cvt_pk_bf16(v[2], v[3])};
  }
}

template <int D, bool Q8>
hipError_t run(const AttnArgs& a, hipStream_t s) {
  const dim3 grid(a.kv_heads, (unsigned)(((int64_t)a.max_q * a.group + 15) / 16), a.seqs);
  attend_rows16_kernel<D, Q8><<<grid, 256, 0, s>>>(a);
  return hipGetLastError();
}

}  // namespace

size_t paged_attention_workspace(const AttnArgs&) { return 0; }

hipError_t launch_paged_attention(const AttnArgs& a, hipStream_t s) {
  const bool q8 = a.scale[0] != nullptr;
  if (a.dim == 64) return q8 ? run<64, true>(a, s) : run<64, false>(a, s);
  return q8 ? run<128, true>(a, s) : run<128, false>(a, s);
}

}  // namespace bd
