// Root-mean-square norm of the residual stream.
//
//   h = x + residual          (float32; written back rounded to bf16)
//   y = h / sqrt(mean(h^2) + eps) * w
//
// y is bf16, or e4m3 with one power-of-two scale per 32 values.  The norm is
// taken of the unrounded float32 sum, so the only roundings are those of the
// outputs.  Bound by HBM: 2 bytes in per value and input, 2 (or 1 + 1/32) out;
// a row stays in registers between its sum of squares and its output, so each
// value is read once: 2048 x 8192 with a residual 21.8 us, 6.2 TB/s with part
// of it in the last-level cache, 25.2 us and 5.3 TB/s from call to call.
#include "common.h"
#include "e4m3.h"
#include "layer.h"

namespace bd {
namespace {

__device__ __forceinline__ u32x4 ld8(const uint16_t* p) {
  return *reinterpret_cast<const u32x4_any*>(p);
}
__device__ __forceinline__ void st8(uint16_t* p, u32x4 v) {
  *reinterpret_cast<u32x4_any*>(p) = v;
}

// Up to eight elements from p, zeros past n.
__device__ __forceinline__ u32x4 ld_some(const uint16_t* p, int n) {
  u32x4 v = {0u, 0u, 0u, 0u};
#pragma unroll
  for (int e = 0; e < 8; ++e)
    if (e < n) v[e >> 1] |= (uint32_t)p[e] << ((e & 1) << 4);
  return v;
}
__device__ __forceinline__ void st_some(uint16_t* p, u32x4 v, int n) {
#pragma unroll
  for (int e = 0; e < 8; ++e)
    if (e < n) p[e] = (uint16_t)(v[e >> 1] >> ((e & 1) << 4));
}

// Sum over the T threads of a row (T = 64, or the whole workgroup).
template <int T>
__device__ __forceinline__ float row_sum(float v, float* red) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o);
  if (T == kWave) return v;
  if ((threadIdx.x & (kWave - 1)) == 0) red[threadIdx.x >> 6] = v;
  __syncthreads();
  float s = 0.f;
#pragma unroll
  for (int i = 0; i < T / kWave; ++i) s += red[i];
  return s;
}

// 1 / sqrt(mean square + eps).  For an 8-bit output as the sum of two floats
// (one Newton step, its products exact by fma), and x times it times w with
// one rounding: next to a border of the group's scale three roundings fall to
// the other side more often, and then the whole group has the other scale.
struct Inv {
  float hi, lo;
};
template <bool MX>
__device__ __forceinline__ Inv inverse(float sum, int cols, float eps) {
  const float a = sum / (float)cols + eps, r = rsqrtf(a);
  if (!MX) return {r, 0.f};
  const float t = a * r;
  const float lo = 0.5f * r * fmaf(-fmaf(a, r, -t), r, fmaf(-t, r, 1.f));
  return {r, fabsf(lo) < INFINITY ? lo : 0.f};
}
template <bool MX>
__device__ __forceinline__ float scaled(float x, Inv i, float w) {
  const float p = x * i.hi;
  if (!MX) return p * w;
  // below 2^-22 of the product; held, so that an infinite w gives infinity
  const float rest = fmaf(x, i.lo, fmaf(x, i.hi, -p)) * w;
  return fmaf(p, w, __builtin_amdgcn_fmed3f(rest, -1e32f, 1e32f));
}

// Eight values of one row: load x (+ residual), write h, keep float32.
template <bool RES>
__device__ __forceinline__ void load_sum(const uint16_t* x, const uint16_t* r, uint16_t* h,
                                         int n, float (&f)[8]) {
  const bool all = n >= 8;
  const u32x4 a = all ? ld8(x) : ld_some(x, n);
#pragma unroll
  for (int d = 0; d < 4; ++d) {
    f[2 * d] = lo16(a[d]);
    f[2 * d + 1] = hi16(a[d]);
  }
  if (RES) {
    const u32x4 b = all ? ld8(r) : ld_some(r, n);
    u32x4 o;
#pragma unroll
    for (int d = 0; d < 4; ++d) {
      f[2 * d] += lo16(b[d]);
      f[2 * d + 1] += hi16(b[d]);
      o[d] = cvt_pk_bf16(f[2 * d], f[2 * d + 1]);
    }
    if (all) st8(h, o);
    else st_some(h, o, n);
  }
}

// Eight normalised values out.  In 8 bits four neighbouring lanes hold a
// group of 32 and share its largest magnitude.
template <bool MX>
__device__ __forceinline__ void put(const NormArgs& a, int64_t row, int col, int n,
                                    const float (&f)[8], Inv inv) {
  const u32x4 w = n >= 8 ? ld8(a.w + col) : ld_some(a.w + col, n);
  float y[8];
#pragma unroll
  for (int d = 0; d < 4; ++d) {
    y[2 * d] = scaled<MX>(f[2 * d], inv, lo16(w[d]));
    y[2 * d + 1] = scaled<MX>(f[2 * d + 1], inv, hi16(w[d]));
  }
  if (!MX) {
    u32x4 o;
#pragma unroll
    for (int d = 0; d < 4; ++d) o[d] = cvt_pk_bf16(y[2 * d], y[2 * d + 1]);
    uint16_t* p = static_cast<uint16_t*>(a.y) + row * a.cols + col;
    if (n >= 8) st8(p, o);
    else st_some(p, o, n);
    return;
  }
  float m = 0.f;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    y[e] = hold_e4m3(y[e]);
    m = fmaxf(m, fabsf(y[e]));
  }
  m = fmaxf(m, __shfl_xor(m, 1));
  m = fmaxf(m, __shfl_xor(m, 2));
  const uint32_t sb = scale_byte(m);
  const float is = inv_scale(sb);
  const u32x2 o = {pack_e4m3(y[0] * is, y[1] * is, y[2] * is, y[3] * is),
                   pack_e4m3(y[4] * is, y[5] * is, y[6] * is, y[7] * is)};
  *reinterpret_cast<u32x2*>(static_cast<uint8_t*>(a.y) + row * a.cols + col) = o;
  if ((threadIdx.x & 3) == 0) a.scale[row * (a.cols >> 5) + (col >> 5)] = (uint8_t)sb;
}

// T threads a row, CH groups of eight values a thread.
template <int T, int CH, bool RES, bool MX>
__global__ __launch_bounds__(T < 256 ? 256 : T) void rms_norm_kernel(const NormArgs a) {
  __shared__ float red[T / kWave];
  const int t = T < 256 ? threadIdx.x & (T - 1) : threadIdx.x;
  const int64_t row = T < 256 ? (int64_t)blockIdx.x * (256 / T) + threadIdx.x / T : blockIdx.x;
  if (T < 256 && row >= a.rows) return;  // whole waves
  const uint16_t* x = a.x + row * a.x_stride;
  const uint16_t* r = RES ? a.residual + row * a.r_stride : nullptr;
  uint16_t* h = RES ? a.h + row * a.cols : nullptr;
  float f[CH][8];
  float ss = 0.f;
#pragma unroll
  for (int c = 0; c < CH; ++c) {
    const int col = (c * T + t) * 8;
#pragma unroll
    for (int e = 0; e < 8; ++e) f[c][e] = 0.f;
    if (col < a.cols) load_sum<RES>(x + col, r + col, h + col, a.cols - col, f[c]);
  }
#pragma unroll
  for (int c = 0; c < CH; ++c)
#pragma unroll
    for (int e = 0; e < 8; ++e) ss = fmaf(f[c][e], f[c][e], ss);
  const Inv inv = inverse<MX>(row_sum<T>(ss, red), a.cols, a.eps);
#pragma unroll
  for (int c = 0; c < CH; ++c) {
    const int col = (c * T + t) * 8;
    if (col < a.cols) put<MX>(a, row, col, a.cols - col, f[c], inv);
  }
}

// Rows too long for the registers of one workgroup: the sum is formed twice.
template <bool RES, bool MX>
__global__ __launch_bounds__(1024) void rms_norm_long_kernel(const NormArgs a) {
  __shared__ float red[16];
  const int64_t row = blockIdx.x;
  const uint16_t* x = a.x + row * a.x_stride;
  const uint16_t* r = RES ? a.residual + row * a.r_stride : nullptr;
  uint16_t* h = RES ? a.h + row * a.cols : nullptr;
  float ss = 0.f;
  float f[8];
  for (int64_t col = threadIdx.x * 8; col < a.cols; col += 8192) {
#pragma unroll
    for (int e = 0; e < 8; ++e) f[e] = 0.f;
    load_sum<RES>(x + col, r + col, h + col, (int)(a.cols - col), f);
#pragma unroll
    for (int e = 0; e < 8; ++e) ss = fmaf(f[e], f[e], ss);
  }
  const Inv inv = inverse<MX>(row_sum<1024>(ss, red), a.cols, a.eps);
  for (int64_t col = threadIdx.x * 8; col < a.cols; col += 8192) {
    load_sum<RES>(x + col, r + col, h + col, (int)(a.cols - col), f);
    put<MX>(a, row, (int)col, (int)(a.cols - col), f, inv);
  }
}

// A launch takes fewer than 2^32 threads: more rows than that go in several,
// of 2^31 threads each.
constexpr int64_t kMostThreads = int64_t(1) << 31;

template <int T, int CH, bool RES, bool MX>
hipError_t rows_of(const NormArgs& a, hipStream_t s) {
  constexpr int kBlock = T < 256 ? 256 : T, kRows = kBlock / T;   // of a workgroup
  constexpr int64_t kMost = kMostThreads / T;
  for (int64_t at = 0; at < a.rows; at += kMost) {
    NormArgs b = a;
    b.rows = a.rows - at < kMost ? a.rows - at : kMost;
    b.x += at * a.x_stride;
    if (RES) b.residual += at * a.r_stride;
    if (RES) b.h += at * a.cols;
    b.y = static_cast<uint8_t*>(a.y) + at * a.cols * (MX ? 1 : 2);
    if (MX) b.scale += at * (a.cols >> 5);
    const unsigned grid = (unsigned)((b.rows + kRows - 1) / kRows);
    if constexpr (CH > 0)
      rms_norm_kernel<T, CH, RES, MX><<<grid, kBlock, 0, s>>>(b);
    else
      rms_norm_long_kernel<RES, MX><<<grid, kBlock, 0, s>>>(b);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

// Threads of a row, by its length.  A wave by itself needs no barrier (20000
// rows of 512: 13.7 us, 256 threads 15.4); more than two groups a thread lose
// loads in flight (8000 rows of 2048: 256 threads 21.0, a wave 23.1; 4096 rows
// of 4096: 512 threads 21.3, a wave 22.3, one row 2.5 and 5.6; 1000 of 16384:
// 1024 threads 23.7, 512 24.8).  A row of 8192 takes 1024 threads (one row 2.9
// us, 512 threads 3.3), for many rows in 8 bits, where the arithmetic counts,
// 512 (2021 rows 20.1, 1024 threads 21.3).
template <bool RES, bool MX>
hipError_t pick(const NormArgs& a, hipStream_t s) {
  if (a.cols <= 512) return rows_of<64, 1, RES, MX>(a, s);
  if (a.cols <= 1024) return rows_of<64, 2, RES, MX>(a, s);
  if (a.cols <= 2048) return rows_of<256, 1, RES, MX>(a, s);
  if (a.cols <= 4096) return rows_of<512, 1, RES, MX>(a, s);
  if (MX && a.cols <= 8192 && a.rows >= 256) return rows_of<512, 2, RES, MX>(a, s);
  if (a.cols <= 8192) return rows_of<1024, 1, RES, MX>(a, s);
  if (a.cols <= 16384) return rows_of<1024, 2, RES, MX>(a, s);
  return rows_of<1024, 0, RES, MX>(a, s);
}

// ------------------------------------------------------------------ around a block
// Eight values of w (1 past the row, where there is no w).
__device__ __forceinline__ void weight8(const uint16_t* w, int n, float (&f)[8]) {
  if (!w) {
#pragma unroll
    for (int e = 0; e < 8; ++e) f[e] = 1.f;
    return;
  }
  const u32x4 v = n >= 8 ? ld8(w) : ld_some(w, n);
#pragma unroll
  for (int d = 0; d < 4; ++d) {
    f[2 * d] = lo16(v[d]);
    f[2 * d + 1] = hi16(v[d]);
  }
}

// h = residual + alpha * gate * x * inv * post, of which x comes in and h goes
// out as float32 and, rounded, to memory.
__device__ __forceinline__ void add_block(const BlockNormArgs& a, int64_t row, int col, int n,
                                          float inv, float (&f)[8]) {
  float p[8], g[8], r[8];
  weight8(a.post ? a.post + col : nullptr, n, p);
  weight8(a.gate ? a.gate + row * a.g_stride + col : nullptr, n, g);
  weight8(a.residual + row * a.r_stride + col, n, r);
  u32x4 o;
#pragma unroll
  for (int e = 0; e < 8; ++e) f[e] = fmaf(f[e] * inv * p[e] * g[e], a.alpha, r[e]);
#pragma unroll
  for (int d = 0; d < 4; ++d) o[d] = cvt_pk_bf16(f[2 * d], f[2 * d + 1]);
  uint16_t* h = a.h + row * a.cols + col;
  if (n >= 8) st8(h, o);
  else st_some(h, o, n);
}

__device__ __forceinline__ void put_block(const BlockNormArgs& a, int64_t row, int col, int n,
                                          float inv, const float (&f)[8]) {
  float w[8];
  weight8(a.w + col, n, w);
  u32x4 o;
#pragma unroll
  for (int d = 0; d < 4; ++d)
    o[d] = cvt_pk_bf16(f[2 * d] * inv * w[2 * d], f[2 * d + 1] * inv * w[2 * d + 1]);
  uint16_t* y = a.y + row * a.cols + col;
  if (n >= 8) st8(y, o);
  else st_some(y, o, n);
}

// The norm after a block and the one before the next: as rms_norm_kernel, with
// a row's x and then its h in registers and a sum of squares of each, so every
// value is read once.  Bound by HBM: 2048 x 8192 with a gate for each value (168
// MB) 33 us, 5.1 TB/s, as a copy; one row 3.4 us.
template <int T, int CH>
__global__ __launch_bounds__(T < 256 ? 256 : T) void rms_norm_block_kernel(const BlockNormArgs a) {
  __shared__ float red[2][T / kWave];
  const int t = T < 256 ? threadIdx.x & (T - 1) : threadIdx.x;
  const int64_t row = T < 256 ? (int64_t)blockIdx.x * (256 / T) + threadIdx.x / T : blockIdx.x;
  if (T < 256 && row >= a.rows) return;  // whole waves
  float f[CH][8];
  float ss = 0.f;
#pragma unroll
  for (int c = 0; c < CH; ++c) {
    const int col = (c * T + t) * 8;
#pragma unroll
    for (int e = 0; e < 8; ++e) f[c][e] = 0.f;
    if (col < a.cols)
      load_sum<false>(a.x + row * a.x_stride + col, nullptr, nullptr, a.cols - col, f[c]);
  }
  float inv = 1.f;
  if (a.post) {   // the same for all
#pragma unroll
    for (int c = 0; c < CH; ++c)
#pragma unroll
      for (int e = 0; e < 8; ++e) ss = fmaf(f[c][e], f[c][e], ss);
    inv = inverse<false>(row_sum<T>(ss, red[0]), a.cols, a.eps).hi;
  }
  ss = 0.f;
#pragma unroll
  for (int c = 0; c < CH; ++c) {
    const int col = (c * T + t) * 8;
    if (col < a.cols) {
      add_block(a, row, col, a.cols - col, inv, f[c]);
#pragma unroll
      for (int e = 0; e < 8; ++e) ss = fmaf(f[c][e], f[c][e], ss);
    }
  }
  inv = inverse<false>(row_sum<T>(ss, red[1]), a.cols, a.eps).hi;
#pragma unroll
  for (int c = 0; c < CH; ++c) {
    const int col = (c * T + t) * 8;
    if (col < a.cols) put_block(a, row, col, a.cols - col, inv, f[c]);
  }
}

// Rows too long for the registers of one workgroup: x is read three times, the
// residual and the gate twice, and h written twice with the same bits.  512 x 32768
// with a gate 48 us, 3.5 TB/s of what is needed (1024 x 16384 26 us, 6.5 with part of
// it in the last-level cache; the residual norm of such rows 3.8).
__global__ __launch_bounds__(1024) void rms_norm_block_long_kernel(const BlockNormArgs a) {
  __shared__ float red[2][16];
  const int64_t row = blockIdx.x;
  const uint16_t* x = a.x + row * a.x_stride;
  float f[8], ss = 0.f, inv = 1.f;
  auto value = [&](int64_t col) {
#pragma unroll
    for (int e = 0; e < 8; ++e) f[e] = 0.f;
    load_sum<false>(x + col, nullptr, nullptr, (int)(a.cols - col), f);
  };
  if (a.post) {
    for (int64_t col = threadIdx.x * 8; col < a.cols; col += 8192) {
      value(col);
#pragma unroll
      for (int e = 0; e < 8; ++e) ss = fmaf(f[e], f[e], ss);
    }
    inv = inverse<false>(row_sum<1024>(ss, red[0]), a.cols, a.eps).hi;
  }
  ss = 0.f;
  for (int64_t col = threadIdx.x * 8; col < a.cols; col += 8192) {
    value(col);
    add_block(a, row, (int)col, (int)(a.cols - col), inv, f);
#pragma unroll
    for (int e = 0; e < 8; ++e) ss = fmaf(f[e], f[e], ss);
  }
  const float inv2 = inverse<false>(row_sum<1024>(ss, red[1]), a.cols, a.eps).hi;
  for (int64_t col = threadIdx.x * 8; col < a.cols; col += 8192) {
    value(col);
    add_block(a, row, (int)col, (int)(a.cols - col), inv, f);   // the same bits again
    put_block(a, row, (int)col, (int)(a.cols - col), inv2, f);
  }
}

template <int T, int CH>
hipError_t blocks_of(const BlockNormArgs& a, hipStream_t s) {
  constexpr int kBlock = T < 256 ? 256 : T, kRows = kBlock / T;   // of a workgroup
  constexpr int64_t kMost = kMostThreads / T;
  for (int64_t at = 0; at < a.rows; at += kMost) {
    BlockNormArgs b = a;
    b.rows = a.rows - at < kMost ? a.rows - at : kMost;
    b.x += at * a.x_stride;
    b.residual += at * a.r_stride;
    if (a.gate) b.gate += at * a.g_stride;
    b.h += at * a.cols;
    b.y += at * a.cols;
    const unsigned grid = (unsigned)((b.rows + kRows - 1) / kRows);
    if constexpr (CH > 0) rms_norm_block_kernel<T, CH><<<grid, kBlock, 0, s>>>(b);
    else rms_norm_block_long_kernel<<<grid, kBlock, 0, s>>>(b);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace

// Threads of a row: as for the norm above.
hipError_t launch_rms_norm_block(const BlockNormArgs& a, hipStream_t s) {
  if (a.cols <= 512) return blocks_of<64, 1>(a, s);
  if (a.cols <= 1024) return blocks_of<64, 2>(a, s);
  if (a.cols <= 2048) return blocks_of<256, 1>(a, s);
  if (a.cols <= 4096) return blocks_of<512, 1>(a, s);
  if (a.cols <= 8192) return blocks_of<1024, 1>(a, s);
  if (a.cols <= 16384) return blocks_of<1024, 2>(a, s);
  return blocks_of<1024, 0>(a, s);
}

hipError_t launch_rms_norm(const NormArgs& a, hipStream_t s) {
  if (a.scale) return a.residual ? pick<true, true>(a, s) : pick<false, true>(a, s);
  return a.residual ? pick<true, false>(a, s) : pick<false, false>(a, s);
}

}  // namespace bd
