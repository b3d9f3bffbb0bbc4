// Rotary positions: rows of bf16 heads turned by the angles of their tokens'
// positions, and the table of cosines and sines that the angles come from.
//
// A rotation reads and writes 2 bytes a value and is bound by HBM (16001 tokens of
// 64 heads of 128 102 us, 5.1 TB/s, as a copy; 2048 12.1 us), or, for few tokens,
// by the launch (2.4 us).  The cosines and sines (float32, 4 bytes a value) are
// read from a table rather than computed: a far position times a frequency
// needs 64 bits to keep the angle's fraction of a turn.
#include "rotary.h"

namespace bd {
namespace {

template <bool INTERLEAVED>
__global__ __launch_bounds__(256) void rotary_kernel(const RotaryArgs a) {
  rotate_unit<INTERLEAVED>(a, (int)(blockIdx.x * 256 + threadIdx.x));
}

// Entry (position, pair) of the table: the angle is taken in 64 bits.
__global__ __launch_bounds__(256) void rotary_table_kernel(const double* frequencies, int pairs,
                                                           int64_t first, int64_t n,
                                                           double magnitude, float* table) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= n) return;
  const int64_t p = i / pairs;
  double s, c;
  sincos((double)(first + p) * frequencies[i - p * pairs], &s, &c);
  reinterpret_cast<float2*>(table)[i] = float2{(float)(c * magnitude), (float)(s * magnitude)};
}

}  // namespace

hipError_t launch_rotary(const RotaryArgs& all, hipStream_t s) {
  RotaryArgs a = all;
  const int64_t per = rotary_plan(a);
  // a launch takes fewer than 2^32 threads, and a thread's index is an int
  const int64_t most = (int64_t(1) << 30) / per;
  for (int64_t at = 0; at < all.tokens; at += most) {
    RotaryArgs b = a;
    b.tokens = all.tokens - at < most ? all.tokens - at : most;
    b.x += at * a.x_token_stride;
    b.out += at * a.out_token_stride;
    b.positions += at;
    const unsigned grid = (unsigned)((b.tokens * per + 255) / 256);
    if (a.interleaved) rotary_kernel<true><<<grid, 256, 0, s>>>(b);
    else rotary_kernel<false><<<grid, 256, 0, s>>>(b);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

hipError_t launch_rotary_table(const double* frequencies, int pairs, int64_t first, int64_t length,
                               double magnitude, float* table, hipStream_t s) {
  const int64_t most = (int64_t(1) << 31) / pairs;
  for (int64_t at = 0; at < length; at += most) {
    const int64_t n = (length - at < most ? length - at : most) * pairs;
    rotary_table_kernel<<<(unsigned)((n + 255) / 256), 256, 0, s>>>(
        frequencies, pairs, first + at, n, magnitude, table + at * pairs * 2);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace bd
