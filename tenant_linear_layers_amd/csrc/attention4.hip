// Attention of new tokens over a paged key/value cache in e2m1: the definition
// of attention.hip's, one wave for a row of q and a head.
#include "common.h"
#include "e2m1.h"
#include "layer.h"

namespace bd {
namespace {

__device__ __forceinline__ float value_of(uint32_t word, int i, uint32_t sb) {
  const uint32_t c = word >> (4 * i);
  const float grid[8] = {0.f, 0.5f, 1.f, 1.5f, 2.f, 3.f, 4.f, 6.f};
  const float scale = sb == kNanScale ? NAN : __uint_as_float(sb ? sb << 23 : 0x400000u);
  const float v = grid[c & 7] * scale;
  return c & 8 ? -v : v;
}

template <int D>
__global__ __launch_bounds__(64) void attend4_kernel(const AttnArgs a) {
  __shared__ float q[D], w[64];
  const int lane = threadIdx.x;
  const int t = blockIdx.x, head = blockIdx.y, kvh = head / a.group;
  int b = -1, q0 = 0, n = 0;
  for (int s = 0; s < a.seqs; ++s) {
    const int lo = min(max(a.cu_q[s], 0), a.tokens), hi = min(max(a.cu_q[s + 1], 0), a.tokens);
    if (t >= lo && t < hi) {
      b = s;
      q0 = lo;
      n = hi - lo;
      break;
    }
  }
  if (b < 0) return;
  const int len = min(max(a.kv_len[b], 0), a.width * a.page);
  const int pos = len - n + (t - q0);
  const int lo = a.window ? max(pos - a.window + 1, 0) : 0;
  for (int d = lane; d < D; d += 64)
    q[d] = __uint_as_float((uint32_t)a.q[t * a.q_token_stride + head * a.q_head_stride + d] << 16);
  __syncthreads();
  float m = -INFINITY, l = 0.f, acc[D / 64];
  for (int k = 0; k < D / 64; ++k) acc[k] = 0.f;
  for (int k0 = lo; k0 <= pos; k0 += 64) {
    const int key = k0 + lane;
    int64_t row = -1;
    float z = -INFINITY;
    if (key <= pos) {
      const int page = a.table[(int64_t)b * a.width + key / a.page];
      if (page >= 0 && page < a.pages) {
        row = ((int64_t)page * a.kv_heads + kvh) * a.page + key % a.page;
        z = 0.f;
        for (int g = 0; g < D / 32; ++g) {
          const uint32_t sb = a.scale[0][row * (D / 32) + g];
          for (int j = 0; j < 4; ++j) {
            const uint32_t word =
                *reinterpret_cast<const uint32_t*>(a.cache[0] + row * (D / 2) + g * 16 + j * 4);
            for (int e = 0; e < 8; ++e) z += value_of(word, e, sb) * q[g * 32 + j * 8 + e];
          }
        }
        z *= a.scale_log2;
      } else {
        z = NAN;
      }
    }
    float top = z;
    for (int o = 32; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor(top, o));
    const float m1 = fmaxf(m, top), ref = m1 == -INFINITY ? 0.f : m1;
    const float f = exp2f(m - ref), p = exp2f(z - ref);
    m = m1;
    float sum = p;
    for (int o = 32; o > 0; o >>= 1) sum += __shfl_xor(sum, o);
    l = l * f + sum;
    w[lane] = p;
    for (int k = 0; k < D / 64; ++k) acc[k] *= f;
    for (int j = 0; j < 64 && k0 + j <= pos; ++j) {
      const int64_t r = __shfl(row, j);
      const float pj = w[j];
      if (r < 0) continue;   // its weight, NaN, is in the sum
      for (int k = 0; k < D / 64; ++k) {
        const int d = 64 * k + lane;
        const uint32_t byte = a.cache[1][r * (D / 2) + d / 2];
        acc[k] += pj * value_of(byte, d & 1, a.scale[1][r * (D / 32) + d / 32]);
      }
    }
  }
  for (int k = 0; k < D / 64; ++k)
    a.out[((int64_t)t * a.heads + head) * D + 64 * k + lane] =
        f32_to_bf16_bits(l == 0.f ? 0.f : acc[k] / l);
}

}  // namespace

hipError_t launch_attention_4bit(const AttnArgs& a, hipStream_t s) {
  const dim3 grid((unsigned)a.tokens, (unsigned)a.heads);
  if (a.dim == 64) attend4_kernel<64><<<grid, 64, 0, s>>>(a);
  else attend4_kernel<128><<<grid, 64, 0, s>>>(a);
  return hipGetLastError();
}

}  // namespace bd
