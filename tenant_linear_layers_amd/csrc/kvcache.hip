// The paged key/value cache: rows [dim] of one head and token, in bf16 or in
// e4m3 with one power-of-two scale per row.
//
// Both kernels move each row once and are bound by HBM (2 bytes a value on
// the bf16 side, 2 or 1 + 1/dim on the cache's) or, for a batch of single
// tokens, by the launch.  dim / 8 neighbouring lanes hold a row: one 16-byte
// access a lane on the bf16 side, and the row's largest magnitude by lane
// exchanges, so a row needs no LDS.  Neighbouring rows of a token are its
// heads, contiguous on the side of the tokens.  64 tokens into 8 bits take 3.3
// us, 2048 5.9 us, 16001 back 20.6 us (4.8 TB/s; a copy reaches 4.9).
#include "common.h"
#include "e4m3.h"
#include "layer.h"

namespace bd {
namespace {

// One lane's place: which cache (0 k, 1 v), token, head and the eight values.
struct Place {
  int which, head, piece;
  int64_t token, row;  // row of the cache, or -1 for a slot outside it
};

template <int D>
__device__ __forceinline__ bool place(const KvArgs& a, Place& p) {
  constexpr int L = D / 8;
  const int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
  const int per = 2 * a.heads * L;
  p.token = i / per;
  if (p.token >= a.tokens) return false;
  const int j = (int)(i - p.token * per);
  p.piece = j % L;
  p.which = j / L >= a.heads;
  p.head = j / L - (p.which ? a.heads : 0);
  const int slot = a.slots[p.token];
  const int page = slot / a.page;
  p.row = slot < 0 || slot >= a.n_slots
              ? -1
              : ((int64_t)page * a.heads + p.head) * a.page + (slot - page * a.page);
  return true;
}

template <int D, bool Q8>
__global__ __launch_bounds__(256) void kv_write_kernel(const KvArgs a) {
  Place p;
  if (!place<D>(a, p) || p.row < 0) return;  // whole rows leave together
  const int w = p.which;
  const u32x4 v = *reinterpret_cast<const u32x4_any*>(
      a.src[w] + p.token * a.token_stride[w] + p.head * a.head_stride[w] + p.piece * 8);
  if (!Q8) {
    *reinterpret_cast<u32x4*>(static_cast<uint16_t*>(a.cache[w]) + p.row * D + p.piece * 8) = v;
    return;
  }
  float f[8], m = 0.f;
#pragma unroll
  for (int d = 0; d < 4; ++d) {
    f[2 * d] = hold_e4m3(lo16(v[d]));
    f[2 * d + 1] = hold_e4m3(hi16(v[d]));
    m = fmaxf(m, fmaxf(fabsf(f[2 * d]), fabsf(f[2 * d + 1])));
  }
#pragma unroll
  for (int o = 1; o < D / 8; o <<= 1) m = fmaxf(m, __shfl_xor(m, o));
  const uint32_t sb = scale_byte(m);
  const float is = inv_scale(sb);
  const u32x2 o = {pack_e4m3(f[0] * is, f[1] * is, f[2] * is, f[3] * is),
                   pack_e4m3(f[4] * is, f[5] * is, f[6] * is, f[7] * is)};
  *reinterpret_cast<u32x2*>(static_cast<uint8_t*>(a.cache[w]) + p.row * D + p.piece * 8) = o;
  if (p.piece == 0) a.scale[w][p.row] = (uint8_t)sb;
}

template <int D, bool Q8>
__global__ __launch_bounds__(256) void kv_read_kernel(const KvArgs a) {
  Place p;
  if (!place<D>(a, p)) return;
  const int w = p.which;
  u32x4 v = {0x7FC07FC0u, 0x7FC07FC0u, 0x7FC07FC0u, 0x7FC07FC0u};  // no such slot: NaN
  if (p.row >= 0) {
    if (Q8) {
      const u32x2 c = *reinterpret_cast<const u32x2*>(static_cast<const uint8_t*>(a.cache[w]) +
                                                      p.row * D + p.piece * 8);
      const float s = __uint_as_float((uint32_t)a.scale[w][p.row] << 23);
      v = u32x4{bf16x2_of_e4m3<false>(c[0], s), bf16x2_of_e4m3<true>(c[0], s),
                bf16x2_of_e4m3<false>(c[1], s), bf16x2_of_e4m3<true>(c[1], s)};
    } else {
      v = *reinterpret_cast<const u32x4*>(static_cast<const uint16_t*>(a.cache[w]) + p.row * D +
                                          p.piece * 8);
    }
  }
  *reinterpret_cast<u32x4*>(a.dst[w] + (p.token * a.heads + p.head) * D + p.piece * 8) = v;
}

// A launch takes fewer than 2^32 threads: more tokens than that go in several
// launches, of 2^31 threads at most.
template <int D, bool Q8, bool WRITE>
hipError_t run(const KvArgs& a, hipStream_t s) {
  const int64_t per = (int64_t)2 * a.heads * (D / 8);   // threads of a token
  const int64_t most = (int64_t(1) << 31) / per;
  for (int64_t at = 0; at < a.tokens; at += most) {
    KvArgs b = a;
    b.tokens = a.tokens - at < most ? a.tokens - at : most;
    b.slots += at;
    for (int w = 0; w < 2; ++w) {
      if (WRITE) b.src[w] += at * a.token_stride[w];
      else b.dst[w] += at * a.heads * D;
    }
    const unsigned grid = (unsigned)((b.tokens * per + 255) / 256);
    if (WRITE) kv_write_kernel<D, Q8><<<grid, 256, 0, s>>>(b);
    else kv_read_kernel<D, Q8><<<grid, 256, 0, s>>>(b);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

template <bool WRITE>
hipError_t pick(const KvArgs& a, hipStream_t s) {
  const bool q8 = a.scale[0] != nullptr;
  if (a.dim == 64) return q8 ? run<64, true, WRITE>(a, s) : run<64, false, WRITE>(a, s);
  return q8 ? run<128, true, WRITE>(a, s) : run<128, false, WRITE>(a, s);
}

}  // namespace

hipError_t launch_kv_write(const KvArgs& a, hipStream_t s) { return pick<true>(a, s); }
hipError_t launch_kv_read(const KvArgs& a, hipStream_t s) { return pick<false>(a, s); }

}  // namespace bd
