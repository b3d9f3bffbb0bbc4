// Launchers of the decoder-layer operators beside the linears: the norm of
// the residual stream, the paged key/value cache and attention over it.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "common.h"

namespace bd {

typedef uint32_t u32x2 __attribute__((__vector_size__(8)));
// 16 bytes at an address aligned to its 2-byte elements only (rows of an odd
// length, strided rows): one load or store of the full width all the same.
typedef u32x4 u32x4_any __attribute__((aligned(2)));

// The two bf16 values of a dword.
__device__ __forceinline__ float lo16(uint32_t v) { return __uint_as_float(v << 16); }
__device__ __forceinline__ float hi16(uint32_t v) { return __uint_as_float(v & 0xFFFF0000u); }

// y = h / sqrt(mean(h^2) + eps) * w of each row, h = x + residual.  scale !=
// nullptr: y is e4m3 with one e8m0 scale per 32 values.
struct NormArgs {
  const uint16_t* x;         // [rows, cols], rows x_stride apart
  const uint16_t* residual;  // the same, r_stride apart, or nullptr
  const uint16_t* w;         // [cols]
  uint16_t* h;               // [rows, cols] or nullptr (no residual)
  void* y;                   // [rows, cols] bf16 or e4m3
  uint8_t* scale;            // [rows, cols / 32] or nullptr
  int64_t x_stride, r_stride;
  int64_t rows;
  int cols;
  float eps;
};
hipError_t launch_rms_norm(const NormArgs& a, hipStream_t stream);

// The norm after a block, its gate and residual, and the norm before the next:
//   u = x / sqrt(mean(x^2) + eps) * post   (post == nullptr: u = x)
//   h = residual + alpha * gate * u        (gate == nullptr: 1)
//   y = h / sqrt(mean(h^2) + eps) * w
struct BlockNormArgs {
  const uint16_t* x;         // [rows, cols], rows x_stride apart
  const uint16_t* residual;  // the same, r_stride apart
  const uint16_t* gate;      // the same, g_stride apart (0: one row for all), or nullptr
  const uint16_t* post;      // [cols] or nullptr
  const uint16_t* w;         // [cols]
  uint16_t* h;               // [rows, cols]
  uint16_t* y;               // [rows, cols]
  int64_t x_stride, r_stride, g_stride;
  int64_t rows;
  int cols;
  float alpha, eps;
};
hipError_t launch_rms_norm_block(const BlockNormArgs& a, hipStream_t stream);

// Division of 0 <= x < 2^31 by a number that the host knows.
struct Divisor {
  uint32_t mul, shift;
  int by;
  __device__ __forceinline__ int of(int x) const {
    return (int)((__umulhi((uint32_t)x, mul) + (uint32_t)x) >> shift);
  }
};
Divisor divisor(int by);

// Rows x [tokens, heads, dim] turned by the angles of their tokens' positions:
// of the first rot dims the pairs (i, i + rot / 2), or (2 i, 2 i + 1)
// interleaved.  out may be x itself.
struct RotaryArgs {
  const uint16_t* x;
  uint16_t* out;
  const int32_t* positions;  // [tokens]
  const float* table;        // [length, rot / 2, 2] cosine, sine
  int64_t x_token_stride, x_head_stride, out_token_stride, out_head_stride;
  int64_t tokens;
  int length, heads, dim, rot;
  bool interleaved;
  // set by the launcher: units of a row, of them with pairs; heads a thread
  int units, turning, each, parts;
  Divisor by_units, by_parts;
};
hipError_t launch_rotary(const RotaryArgs& a, hipStream_t stream);
hipError_t launch_rotary_table(const double* frequencies, int pairs, int64_t first, int64_t length,
                               double magnitude, float* table, hipStream_t stream);

// Rows of the cache at `slots`.  Caches are [pages, heads, page, dim]; slot s
// is row s % page of page s / page.  bits: 16 (bf16), 8 (e4m3, a scale a row)
// or 4 (e2m1, a scale for 32 dims of a row).
struct KvArgs {
  const uint16_t* src[2];    // write: k, v [tokens, heads, dim] with strides
  uint16_t* dst[2];          // read: k, v [tokens, heads, dim]
  void* cache[2];
  uint8_t* scale[2];         // e8m0 [pages, heads, page (, dim / 32)], nullptr for bf16
  const int32_t* slots;      // [tokens]
  int64_t token_stride[2], head_stride[2];
  int64_t tokens, n_slots;
  int heads, dim, page, bits;
  Divisor by_token, by_page;   // threads of a token, page (set by the launcher)
};
hipError_t launch_kv_write(const KvArgs& a, hipStream_t stream);
hipError_t launch_kv_read(const KvArgs& a, hipStream_t stream);
// Queries turned (q.x to q.out), and the rows of a kv_write with k turned by
// the same positions and table.
hipError_t launch_kv_append(const KvArgs& a, const RotaryArgs& q, hipStream_t stream);

struct AttnArgs {
  const uint16_t* q;         // [tokens, heads, dim] with strides
  const uint8_t* cache[2];   // k, v: [pages, kv_heads, page, dim]
  const uint8_t* scale[2];   // e8m0 [pages, kv_heads, page (, dim / 32)], nullptr for bf16
  const int32_t* table;      // [seqs, width] page ids
  const int32_t* cu_q;       // [seqs + 1]
  const int32_t* kv_len;     // [seqs]
  uint16_t* out;             // [tokens, heads, dim]
  float* partial;            // workspace
  int64_t q_token_stride, q_head_stride;
  int64_t pages;
  int first;                 // piece of a launch's first workgroup (set by the launcher)
  int tokens, seqs, max_q, heads, kv_heads, group, dim, page, width;
  int bits;                  // of a cached value: 16, 8 or 4
  Divisor by_group, by_page, by_heads;   // group, page, kv_heads (set by the launcher)
  int window;                // 0: none
  int items;                 // pieces that the workspace has room for (set by the launcher)
  float scale_log2;          // softmax scale * log2(e)
};
size_t paged_attention_workspace(const AttnArgs& a);
hipError_t launch_paged_attention(const AttnArgs& a, hipStream_t stream);
hipError_t launch_attention_4bit(const AttnArgs& a, hipStream_t stream);

}  // namespace bd
