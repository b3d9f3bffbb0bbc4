// C ABI of libbitdelta: argument checks, device check and kernel dispatch.
// Every check runs on the host before anything is enqueued; see
// include/bitdelta.h for the contract of each entry point.
#include <atomic>
#include <cmath>
#include <cstring>
#include <mutex>

#include "bitdelta.h"
#include "common.h"
#include "internal.h"
#include "layer.h"
#include "probe.h"
#include "scale_round.h"

#define BD_EXPORT extern "C" __attribute__((visibility("default")))

namespace {

constexpr int64_t kInt32Max = 2147483647;
constexpr int64_t kMaxElems = int64_t(1) << 40;
// The MonoSoup merge kernel's grid takes 64 rows per workgroup in its y
// dimension (at most 65535 workgroups).
constexpr int64_t kMonosoupMaxRows = 65535 * 64;
// The product Delta X addresses a workgroup's 64 rows of each matrix with
// 32-bit buffer offsets: 64 d_in bf16 values must stay below 2 GiB.
constexpr int64_t kMonosoupMaxCols = (int64_t(1) << 24) - 64;

// Row lengths up to 2^30 keep every per-row element and chunk index of the
// kernels (a row's chunks of 512 elements, rounded up) inside a 32-bit int.
constexpr int64_t kMaxDin = int64_t(1) << 30;

bool shape_ok(int64_t d_out, int64_t d_in) {
  return d_out >= 1 && d_in >= 64 && d_in % 64 == 0 && d_out <= kInt32Max && d_in <= kMaxDin &&
         d_out * d_in < kMaxElems;
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

bool overlap(const void* a, size_t na, const void* b, size_t nb) {
  const uintptr_t a0 = reinterpret_cast<uintptr_t>(a), b0 = reinterpret_cast<uintptr_t>(b);
  return a0 < b0 + nb && b0 < a0 + na;
}

// 0 unknown, 1 gfx950, 2 other.  Cached per device index.
std::atomic<int> g_arch_state[64];

int check_device() {
  int dev = 0;
  if (hipGetDevice(&dev) != hipSuccess) return BITDELTA_ERR_HIP;
  if (dev < 0 || dev >= 64) return BITDELTA_ERR_DEVICE;
  int st = g_arch_state[dev].load(std::memory_order_relaxed);
  if (st == 0) {
    hipDeviceProp_t prop;
    if (hipGetDeviceProperties(&prop, dev) != hipSuccess) return BITDELTA_ERR_HIP;
    st = std::strncmp(prop.gcnArchName, "gfx950", 6) == 0 ? 1 : 2;
    g_arch_state[dev].store(st, std::memory_order_relaxed);
  }
  return st == 1 ? BITDELTA_OK : BITDELTA_ERR_DEVICE;
}

int status_of(hipError_t e) { return e == hipSuccess ? BITDELTA_OK : BITDELTA_ERR_HIP; }

}  // namespace

BD_EXPORT const char* bitdelta_status_string(int status) {
  switch (status) {
    case BITDELTA_OK: return "ok";
    case BITDELTA_ERR_NULL: return "a required pointer is NULL";
    case BITDELTA_ERR_SHAPE:
      return "shape out of range (linears: need M >= 1, d_out >= 1, d_in >= 64, d_in % 64 == 0, "
             "each below 2^31, d_out*d_in below 2^40; other calls: the limits of their entry)";
    case BITDELTA_ERR_ALIGN: return "a buffer is not 16-byte aligned";
    case BITDELTA_ERR_MODE: return "alpha_mode must be 0 (per matrix) or 1 (per row)";
    case BITDELTA_ERR_VARIANTS: return "n_variants must be in [1, 64]";
    case BITDELTA_ERR_WORKSPACE: return "workspace missing or too small";
    case BITDELTA_ERR_HIP: return "HIP runtime error";
    case BITDELTA_ERR_DEVICE: return "current device is not a gfx950 GPU";
    case BITDELTA_ERR_OVERLAP: return "an output buffer overlaps an input buffer";
    case BITDELTA_ERR_CACHE:
      return "delta cache: parameter or variant out of range, or call out of order";
    default: return "unknown status";
  }
}

BD_EXPORT uint32_t bitdelta_ratio_to_f32_bits(uint64_t s_hi, uint64_t s_lo, uint64_t n) {
  return bd::ratio_to_f32_bits(s_hi, s_lo, n);
}

BD_EXPORT size_t bitdelta_compress_workspace_size(int64_t d_out, int64_t d_in, int alpha_mode) {
  if (!shape_ok(d_out, d_in)) return 0;
  if (alpha_mode == BITDELTA_ALPHA_PER_MATRIX) return (size_t)d_out * 16u;
  return 0;
}

BD_EXPORT int bitdelta_compress(const uint16_t* w_ft, const uint16_t* w_base, int64_t d_out,
                                int64_t d_in, int alpha_mode, uint64_t* packed, float* alpha,
                                void* workspace, size_t workspace_bytes, void* stream) {
  if (!w_ft || !w_base || !packed || !alpha) return BITDELTA_ERR_NULL;
  if (!shape_ok(d_out, d_in)) return BITDELTA_ERR_SHAPE;
  if (alpha_mode != BITDELTA_ALPHA_PER_MATRIX && alpha_mode != BITDELTA_ALPHA_PER_ROW)
    return BITDELTA_ERR_MODE;
  if (!aligned16(w_ft) || !aligned16(w_base) || !aligned16(packed) || !aligned16(alpha))
    return BITDELTA_ERR_ALIGN;
  const size_t need = bitdelta_compress_workspace_size(d_out, d_in, alpha_mode);
  if (need > 0 && (!workspace || workspace_bytes < need)) return BITDELTA_ERR_WORKSPACE;
  if (need > 0 && !aligned16(workspace)) return BITDELTA_ERR_ALIGN;
  const size_t wbytes = (size_t)d_out * (size_t)d_in * 2u;
  const size_t pbytes = wbytes / 16u;
  const size_t abytes = alpha_mode == BITDELTA_ALPHA_PER_ROW ? (size_t)d_out * 4u : 4u;
  if (overlap(packed, pbytes, w_ft, wbytes) || overlap(packed, pbytes, w_base, wbytes) ||
      overlap(alpha, abytes, w_ft, wbytes) || overlap(alpha, abytes, w_base, wbytes) ||
      overlap(alpha, abytes, packed, pbytes) ||
      (need > 0 && (overlap(workspace, need, w_ft, wbytes) ||
                    overlap(workspace, need, w_base, wbytes) ||
                    overlap(workspace, need, packed, pbytes) ||
                    overlap(workspace, need, alpha, abytes))))
    return BITDELTA_ERR_OVERLAP;
  const int dev = check_device();
  if (dev != BITDELTA_OK) return dev;
  return status_of(bd::launch_compress(w_ft, w_base, (int)d_out, (int)d_in,
                                       alpha_mode == BITDELTA_ALPHA_PER_ROW, packed, alpha,
                                       static_cast<uint64_t*>(workspace),
                                       static_cast<hipStream_t>(stream)));
}

// ------------------------------------------------------------------ no-alloc
// Scratch of bitdelta_compress_noalloc: the per-row integer partial sums of a
// per-matrix scale (16 bytes per row), in a file-scope device array instead
// of a caller workspace.  Each GPU holds its own copy for the life of the
// process.  Host code never uses the array's name as an address: the device
// address is looked up once per device, with that device current, and kept.
constexpr int64_t kNoAllocMaxRows = 262144;  // 4 MiB of scratch
static __device__ __align__(256) uint64_t scratch[2 * kNoAllocMaxRows];

namespace {
void* g_scratch_ptr[64];
hipError_t g_scratch_err[64];
std::once_flag g_scratch_once[64];

// Device address of this device's scratch (nullptr on failure, with *err set).
void* scratch_on_current_device(hipError_t* err) {
  int dev = 0;
  *err = hipGetDevice(&dev);
  if (*err != hipSuccess) return nullptr;
  if (dev < 0 || dev >= 64) {
    *err = hipErrorInvalidDevice;
    return nullptr;
  }
  std::call_once(g_scratch_once[dev], [dev] {
    void* p = nullptr;
    const hipError_t e = hipGetSymbolAddress((void**)&p, HIP_SYMBOL(scratch));
    g_scratch_err[dev] = e;
    g_scratch_ptr[dev] = e == hipSuccess ? p : nullptr;
  });
  *err = g_scratch_err[dev];
  return g_scratch_ptr[dev];
}
}  // namespace

BD_EXPORT int bitdelta_compress_noalloc(const uint16_t* w_ft, const uint16_t* w_base,
                                        int64_t d_out, int64_t d_in, int alpha_mode,
                                        uint64_t* packed, float* alpha, void* stream) {
  if (!w_ft || !w_base || !packed || !alpha) return BITDELTA_ERR_NULL;
  if (!shape_ok(d_out, d_in)) return BITDELTA_ERR_SHAPE;
  if (alpha_mode != BITDELTA_ALPHA_PER_MATRIX && alpha_mode != BITDELTA_ALPHA_PER_ROW)
    return BITDELTA_ERR_MODE;
  if (alpha_mode == BITDELTA_ALPHA_PER_MATRIX && d_out > kNoAllocMaxRows)
    return BITDELTA_ERR_WORKSPACE;
  if (!aligned16(w_ft) || !aligned16(w_base) || !aligned16(packed) || !aligned16(alpha))
    return BITDELTA_ERR_ALIGN;
  const size_t wbytes = (size_t)d_out * (size_t)d_in * 2u;
  const size_t pbytes = wbytes / 16u;
  const size_t abytes = alpha_mode == BITDELTA_ALPHA_PER_ROW ? (size_t)d_out * 4u : 4u;
  if (overlap(packed, pbytes, w_ft, wbytes) || overlap(packed, pbytes, w_base, wbytes) ||
      overlap(alpha, abytes, w_ft, wbytes) || overlap(alpha, abytes, w_base, wbytes) ||
      overlap(alpha, abytes, packed, pbytes))
    return BITDELTA_ERR_OVERLAP;
  const int dev = check_device();
  if (dev != BITDELTA_OK) return dev;
  uint64_t* partial = nullptr;
  if (alpha_mode == BITDELTA_ALPHA_PER_MATRIX) {
    hipError_t e = hipSuccess;
    partial = static_cast<uint64_t*>(scratch_on_current_device(&e));
    if (e != hipSuccess || !partial) return BITDELTA_ERR_HIP;
  }
  // The row pass writes both limbs of every row 0..d_out-1 before the
  // finalize reads them, so nothing left by an earlier call is ever read.
  return status_of(bd::launch_compress(w_ft, w_base, (int)d_out, (int)d_in,
                                       alpha_mode == BITDELTA_ALPHA_PER_ROW, packed, alpha,
                                       partial, static_cast<hipStream_t>(stream)));
}

BD_EXPORT int bitdelta_linear(const uint16_t* x, int64_t M, const uint16_t* w_base,
                              const uint64_t* packed, const float* alpha, int alpha_mode,
                              int64_t d_out, int64_t d_in, uint16_t* y, void* stream) {
  if (!x || !w_base || !packed || !alpha || !y) return BITDELTA_ERR_NULL;
  if (!shape_ok(d_out, d_in) || M < 1 || M > kInt32Max || M * d_in >= kMaxElems ||
      M * d_out >= kMaxElems ||
      d_in > (M > bd::kMaxSkinnyTokens ? bd::kPrefillMaxDin : bd::kSkinnyMaxDin))
    return BITDELTA_ERR_SHAPE;
  if (alpha_mode != BITDELTA_ALPHA_PER_MATRIX && alpha_mode != BITDELTA_ALPHA_PER_ROW)
    return BITDELTA_ERR_MODE;
  if (!aligned16(x) || !aligned16(w_base) || !aligned16(packed) || !aligned16(y))
    return BITDELTA_ERR_ALIGN;
  if (reinterpret_cast<uintptr_t>(alpha) & 3u) return BITDELTA_ERR_ALIGN;
  const size_t ybytes = (size_t)M * (size_t)d_out * 2u;
  const size_t wbytes = (size_t)d_out * (size_t)d_in * 2u;
  const size_t abytes = alpha_mode == BITDELTA_ALPHA_PER_ROW ? (size_t)d_out * 4u : 4u;
  if (overlap(y, ybytes, x, (size_t)M * (size_t)d_in * 2u) || overlap(y, ybytes, w_base, wbytes) ||
      overlap(y, ybytes, packed, wbytes / 16u) || overlap(y, ybytes, alpha, abytes))
    return BITDELTA_ERR_OVERLAP;
  const int dev = check_device();
  if (dev != BITDELTA_OK) return dev;
  hipStream_t s = static_cast<hipStream_t>(stream);
  if (M <= bd::kMaxSkinnyTokens) {
    bd::SkinnyArgs a;
    std::memset(&a, 0, sizeof(a));
    a.x = x;
    a.ids = nullptr;
    a.w = w_base;
    a.y = y;
    a.M = (int)M;
    a.d_out = (int)d_out;
    a.d_in = (int)d_in;
    a.per_row = alpha_mode == BITDELTA_ALPHA_PER_ROW;
    a.n_variants = 1;
    a.packed[0] = reinterpret_cast<const uint32_t*>(packed);
    a.alpha[0] = alpha;
    return status_of(bd::launch_linear_skinny(a, s));
  }
  return status_of(bd::launch_linear_prefill(
      x, (int)M, w_base, reinterpret_cast<const uint8_t*>(packed), alpha,
      alpha_mode == BITDELTA_ALPHA_PER_ROW, (int)d_out, (int)d_in, y, s));
}

BD_EXPORT int bitdelta_linear_multi(const uint16_t* x, int64_t M, const int32_t* variant_ids,
                                    const uint16_t* w_base, int32_t n_variants,
                                    const uint64_t* const* packed, const float* const* alpha,
                                    int alpha_mode, int64_t d_out, int64_t d_in, uint16_t* y,
                                    void* stream) {
  if (!x || !variant_ids || !w_base || !packed || !alpha || !y) return BITDELTA_ERR_NULL;
  if (!shape_ok(d_out, d_in) || M < 1 || M > kInt32Max || M * d_in >= kMaxElems ||
      M * d_out >= kMaxElems || d_in > bd::kSkinnyMaxDin)
    return BITDELTA_ERR_SHAPE;
  if (alpha_mode != BITDELTA_ALPHA_PER_MATRIX && alpha_mode != BITDELTA_ALPHA_PER_ROW)
    return BITDELTA_ERR_MODE;
  if (n_variants < 1 || n_variants > BITDELTA_MAX_VARIANTS) return BITDELTA_ERR_VARIANTS;
  for (int v = 0; v < n_variants; ++v)
    if (!packed[v] || !alpha[v]) return BITDELTA_ERR_NULL;
  if (!aligned16(x) || !aligned16(w_base) || !aligned16(y) ||
      (reinterpret_cast<uintptr_t>(variant_ids) & 3u))
    return BITDELTA_ERR_ALIGN;
  for (int v = 0; v < n_variants; ++v)
    if (!aligned16(packed[v]) || (reinterpret_cast<uintptr_t>(alpha[v]) & 3u))
      return BITDELTA_ERR_ALIGN;
  const size_t ybytes = (size_t)M * (size_t)d_out * 2u;
  const size_t wbytes = (size_t)d_out * (size_t)d_in * 2u;
  const size_t abytes = alpha_mode == BITDELTA_ALPHA_PER_ROW ? (size_t)d_out * 4u : 4u;
  if (overlap(y, ybytes, x, (size_t)M * (size_t)d_in * 2u) || overlap(y, ybytes, w_base, wbytes) ||
      overlap(y, ybytes, variant_ids, (size_t)M * 4u))
    return BITDELTA_ERR_OVERLAP;
  for (int v = 0; v < n_variants; ++v)
    if (overlap(y, ybytes, packed[v], wbytes / 16u) || overlap(y, ybytes, alpha[v], abytes))
      return BITDELTA_ERR_OVERLAP;
  const int dev = check_device();
  if (dev != BITDELTA_OK) return dev;
  hipStream_t s = static_cast<hipStream_t>(stream);
  bd::SkinnyArgs a;
  std::memset(&a, 0, sizeof(a));
  a.w = w_base;
  a.d_out = (int)d_out;
  a.d_in = (int)d_in;
  a.per_row = alpha_mode == BITDELTA_ALPHA_PER_ROW;
  a.n_variants = n_variants;
  for (int v = 0; v < n_variants; ++v) {
    a.packed[v] = reinterpret_cast<const uint32_t*>(packed[v]);
    a.alpha[v] = alpha[v];
  }
  for (int64_t m0 = 0; m0 < M; m0 += bd::kMaxSkinnyTokens) {
    const int mc = (int)((M - m0) < bd::kMaxSkinnyTokens ? (M - m0) : bd::kMaxSkinnyTokens);
    a.x = x + m0 * d_in;
    a.ids = variant_ids + m0;
    a.y = y + m0 * d_out;
    a.M = mc;
    const int st = status_of(bd::launch_linear_multi(a, s));
    if (st != BITDELTA_OK) return st;
  }
  return BITDELTA_OK;
}

BD_EXPORT int bitdelta_reconstruct(const uint16_t* w_base, const uint64_t* packed,
                                   const float* alpha, int alpha_mode, int64_t d_out,
                                   int64_t d_in, uint16_t* w_eff, void* stream) {
  if (!w_base || !packed || !alpha || !w_eff) return BITDELTA_ERR_NULL;
  if (!shape_ok(d_out, d_in)) return BITDELTA_ERR_SHAPE;
  if (alpha_mode != BITDELTA_ALPHA_PER_MATRIX && alpha_mode != BITDELTA_ALPHA_PER_ROW)
    return BITDELTA_ERR_MODE;
  if (!aligned16(w_base) || !aligned16(packed) || !aligned16(w_eff)) return BITDELTA_ERR_ALIGN;
  if (reinterpret_cast<uintptr_t>(alpha) & 3u) return BITDELTA_ERR_ALIGN;
  const size_t wbytes = (size_t)d_out * (size_t)d_in * 2u;
  const size_t abytes = alpha_mode == BITDELTA_ALPHA_PER_ROW ? (size_t)d_out * 4u : 4u;
  if (overlap(w_eff, wbytes, w_base, wbytes) || overlap(w_eff, wbytes, packed, wbytes / 16u) ||
      overlap(w_eff, wbytes, alpha, abytes))
    return BITDELTA_ERR_OVERLAP;
  const int dev = check_device();
  if (dev != BITDELTA_OK) return dev;
  return status_of(bd::launch_reconstruct(w_base, reinterpret_cast<const uint8_t*>(packed), alpha,
                                          alpha_mode == BITDELTA_ALPHA_PER_ROW, (int)d_out,
                                          (int)d_in, w_eff, static_cast<hipStream_t>(stream)));
}

BD_EXPORT size_t bitdelta_monosoup_workspace_size(int64_t d_out, int64_t d_in, int32_t k,
                                                  int32_t rank) {
  if (!shape_ok(d_out, d_in) || k < 1 || k > BITDELTA_MONOSOUP_MAX_CHECKPOINTS || rank < 1 ||
      rank > BITDELTA_MONOSOUP_MAX_RANK || rank > d_out || rank > d_in ||
      d_out > kMonosoupMaxRows || d_in > kMonosoupMaxCols)
    return 0;
  return bd::monosoup_workspace_bytes(d_out, d_in, k, rank);
}

BD_EXPORT int bitdelta_monosoup_merge(const uint16_t* const* w_ft, int32_t k,
                                      const uint16_t* w_base, int64_t d_out, int64_t d_in,
                                      int32_t rank, int32_t power_iters, const float* omega,
                                      uint16_t* w_merged, float* tau_mean, void* workspace,
                                      size_t workspace_bytes, void* stream) {
  if (!w_ft || !w_base || !omega || !w_merged || !workspace) return BITDELTA_ERR_NULL;
  if (!shape_ok(d_out, d_in) || k < 1 || k > BITDELTA_MONOSOUP_MAX_CHECKPOINTS || rank < 1 ||
      rank > BITDELTA_MONOSOUP_MAX_RANK || rank > d_out || rank > d_in || power_iters < 0 ||
      power_iters > BITDELTA_MONOSOUP_MAX_POWER_ITERS || d_out * d_in >= kMaxElems / 4 ||
      d_out > kMonosoupMaxRows || d_in > kMonosoupMaxCols)
    return BITDELTA_ERR_SHAPE;
  for (int i = 0; i < k; ++i)
    if (!w_ft[i]) return BITDELTA_ERR_NULL;
  for (int i = 0; i < k; ++i)
    if (!aligned16(w_ft[i])) return BITDELTA_ERR_ALIGN;
  if (!aligned16(w_base) || !aligned16(w_merged) || !aligned16(workspace) ||
      (tau_mean && !aligned16(tau_mean)) || (reinterpret_cast<uintptr_t>(omega) & 3u))
    return BITDELTA_ERR_ALIGN;
  const size_t need = bd::monosoup_workspace_bytes(d_out, d_in, k, rank);
  if (workspace_bytes < need) return BITDELTA_ERR_WORKSPACE;
  const size_t wbytes = (size_t)d_out * (size_t)d_in * 2u;
  const size_t tbytes = wbytes * 2u;
  const size_t obytes = (size_t)d_in * (size_t)rank * 4u;
  const void* outs[3] = {w_merged, tau_mean, workspace};
  const size_t outn[3] = {wbytes, tbytes, need};
  for (int a = 0; a < 3; ++a) {
    if (!outs[a]) continue;
    if (overlap(outs[a], outn[a], w_base, wbytes) || overlap(outs[a], outn[a], omega, obytes))
      return BITDELTA_ERR_OVERLAP;
    for (int i = 0; i < k; ++i)
      if (overlap(outs[a], outn[a], w_ft[i], wbytes)) return BITDELTA_ERR_OVERLAP;
    for (int b = a + 1; b < 3; ++b)
      if (outs[b] && overlap(outs[a], outn[a], outs[b], outn[b])) return BITDELTA_ERR_OVERLAP;
  }
  const int dev = check_device();
  if (dev != BITDELTA_OK) return dev;
  return status_of(bd::launch_monosoup(w_ft, k, w_base, (int)d_out, (int)d_in, rank, power_iters,
                                       omega, w_merged, tau_mean, workspace,
                                       static_cast<hipStream_t>(stream)));
}

// ------------------------------------------------------------------ layer operators
namespace {

bool aligned2(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 1u) == 0; }
bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

// Bytes from the first to past the last element of a strided bf16 tensor.
size_t span(int64_t n0, int64_t s0, int64_t n1, int64_t s1, int64_t inner) {
  return (size_t)((n0 - 1) * s0 + (n1 - 1) * s1 + inner) * 2u;
}

int rms_norm(const uint16_t* x, int64_t x_stride, const uint16_t* residual, int64_t r_stride,
             const uint16_t* w, float eps, int64_t rows, int64_t cols, uint16_t* h_out, void* y,
             uint8_t* scale, bool mx, void* stream) {
  if (rows < 0 || rows > kInt32Max || cols < 1 || cols > kMaxDin || rows * cols >= kMaxElems ||
      (mx && cols % 32 != 0))
    return BITDELTA_ERR_SHAPE;
  if (rows == 0) return BITDELTA_OK;
  if (!x || !w || !y || (residual != nullptr) != (h_out != nullptr) || (mx && !scale))
    return BITDELTA_ERR_NULL;
  if (x_stride < 0 || (residual && r_stride < 0) || x_stride >= kMaxElems ||
      (residual && r_stride >= kMaxElems))
    return BITDELTA_ERR_SHAPE;
  if (!aligned2(x) || !aligned2(w) || !aligned2(residual) || !aligned2(h_out) ||
      (mx ? !aligned16(y) : !aligned2(y)))
    return BITDELTA_ERR_ALIGN;
  const size_t n = (size_t)rows * (size_t)cols;
  const void* outs[3] = {y, h_out, scale};
  const size_t outn[3] = {mx ? n : 2 * n, 2 * n, n / 32};
  const void* ins[3] = {x, residual, w};
  const size_t inn[3] = {span(rows, x_stride, 1, 0, cols), span(rows, r_stride, 1, 0, cols),
                         (size_t)cols * 2u};
  for (int i = 0; i < 3; ++i) {
    if (!outs[i]) continue;
    for (int j = 0; j < 3; ++j)
      if (ins[j] && overlap(outs[i], outn[i], ins[j], inn[j])) return BITDELTA_ERR_OVERLAP;
    for (int j = i + 1; j < 3; ++j)
      if (outs[j] && overlap(outs[i], outn[i], outs[j], outn[j])) return BITDELTA_ERR_OVERLAP;
  }
  const int dev = check_device();
  if (dev != BITDELTA_OK) return dev;
  bd::NormArgs a{};
  a.x = x;
  a.residual = residual;
  a.w = w;
  a.h = h_out;
  a.y = y;
  a.scale = scale;
  a.x_stride = x_stride;
  a.r_stride = r_stride;
  a.rows = rows;
  a.cols = (int)cols;
  a.eps = eps;
  return status_of(bd::launch_rms_norm(a, static_cast<hipStream_t>(stream)));
}

bool cache_shape_ok(int64_t heads, int64_t dim, int64_t pages, int64_t page) {
  return heads >= 1 && heads <= 1024 && (dim == 64 || dim == 128) && page >= 16 &&
         page % 16 == 0 && page <= 65536 && pages >= 1 && pages <= kInt32Max / page &&
         pages * page <= (int64_t(1) << 35) / heads;  // groups of 16 rows count in an int
}

}  // namespace

BD_EXPORT int bitdelta_rms_norm(const uint16_t* x, int64_t x_stride, const uint16_t* residual,
                                int64_t r_stride, const uint16_t* w, float eps, int64_t rows,
                                int64_t cols, uint16_t* h_out, uint16_t* y, void* stream) {
  return rms_norm(x, x_stride, residual, r_stride, w, eps, rows, cols, h_out, y, nullptr, false,
                  stream);
}

BD_EXPORT int bitdelta_rms_norm_mx(const uint16_t* x, int64_t x_stride, const uint16_t* residual,
                                   int64_t r_stride, const uint16_t* w, float eps, int64_t rows,
                                   int64_t cols, uint16_t* h_out, uint8_t* y, uint8_t* scale,
                                   void* stream) {
  return rms_norm(x, x_stride, residual, r_stride, w, eps, rows, cols, h_out, y, scale, true,
                  stream);
}

namespace {

// Bytes of a cache's rows, and of their scales, in bf16, e4m3 or e2m1.
size_t cache_bytes(size_t rows, int64_t dim, int bits) {
  return rows * (size_t)dim * (size_t)bits / 8u;
}
size_t scale_bytes(size_t rows, int64_t dim, int bits) {
  return bits == 4 ? rows * (size_t)(dim / 32) : rows;
}
// Scales are there as the format wants them: for 8 bits as k_scale says.
bool scales_ok(const uint8_t* k_scale, const uint8_t* v_scale, int bits) {
  return (k_scale != nullptr) == (bits != 16) && (v_scale != nullptr) == (bits != 16);
}

bool strides_ok(int64_t a, int64_t b) {
  return a >= 0 && b >= 0 && a < kMaxElems && b < kMaxElems;
}

// Everything of a call that puts rows into a cache, its inputs' checks but for
// those of an append's.
int kv_write_args(const uint16_t* k, const uint16_t* v, const int64_t (&strides)[4],
                  const int32_t* slots, int64_t tokens, int64_t heads, int64_t dim, int64_t pages,
                  int64_t page, int bits, void* k_cache, void* v_cache, uint8_t* k_scale,
                  uint8_t* v_scale, bd::KvArgs& a) {
  if (!cache_shape_ok(heads, dim, pages, page) || tokens < 0 || tokens > kInt32Max ||
      tokens * heads * dim >= kMaxElems)
    return BITDELTA_ERR_SHAPE;
  if (!strides_ok(strides[0], strides[1]) || !strides_ok(strides[2], strides[3]))
    return BITDELTA_ERR_SHAPE;
  if (tokens == 0) return BITDELTA_OK;
  if (!k || !v || !slots || !k_cache || !v_cache || !scales_ok(k_scale, v_scale, bits))
    return BITDELTA_ERR_NULL;
  if (!aligned2(k) || !aligned2(v) || !aligned4(slots) || !aligned16(k_cache) ||
      !aligned16(v_cache) || !aligned16(k_scale) || !aligned16(v_scale))
    return BITDELTA_ERR_ALIGN;
  const size_t rows = (size_t)pages * (size_t)page * (size_t)heads;
  const size_t cbytes = cache_bytes(rows, dim, bits), sbytes = scale_bytes(rows, dim, bits);
  const void* outs[4] = {k_cache, v_cache, k_scale, v_scale};
  const size_t outn[4] = {cbytes, cbytes, sbytes, sbytes};
  const void* ins[3] = {k, v, slots};
  const size_t inn[3] = {span(tokens, strides[0], heads, strides[1], dim),
                         span(tokens, strides[2], heads, strides[3], dim), (size_t)tokens * 4u};
  for (int i = 0; i < 4; ++i) {
    if (!outs[i]) continue;
    for (int j = 0; j < 3; ++j)
      if (overlap(outs[i], outn[i], ins[j], inn[j])) return BITDELTA_ERR_OVERLAP;
    for (int j = i + 1; j < 4; ++j)
      if (outs[j] && overlap(outs[i], outn[i], outs[j], outn[j])) return BITDELTA_ERR_OVERLAP;
  }
  a.src[0] = k;
  a.src[1] = v;
  a.cache[0] = k_cache;
  a.cache[1] = v_cache;
  a.scale[0] = k_scale;
  a.scale[1] = v_scale;
  a.slots = slots;
  a.token_stride[0] = strides[0];
  a.token_stride[1] = strides[2];
  a.head_stride[0] = strides[1];
  a.head_stride[1] = strides[3];
  a.tokens = tokens;
  a.n_slots = pages * page;
  a.heads = (int)heads;
  a.dim = (int)dim;
  a.page = (int)page;
  a.bits = bits;
  return BITDELTA_OK;
}

int kv_write(const uint16_t* k, const uint16_t* v, const int64_t (&strides)[4],
             const int32_t* slots, int64_t tokens, int64_t heads, int64_t dim, int64_t pages,
             int64_t page, int bits, void* k_cache, void* v_cache, uint8_t* k_scale,
             uint8_t* v_scale, void* stream) {
  bd::KvArgs a{};
  const int st = kv_write_args(k, v, strides, slots, tokens, heads, dim, pages, page, bits,
                               k_cache, v_cache, k_scale, v_scale, a);
  if (st != BITDELTA_OK || tokens == 0) return st;
  const int dev = check_device();
  if (dev != BITDELTA_OK) return dev;
  return status_of(bd::launch_kv_write(a, static_cast<hipStream_t>(stream)));
}

int kv_read(const int32_t* slots, int64_t tokens, int64_t heads, int64_t dim, int64_t pages,
            int64_t page, int bits, const void* k_cache, const void* v_cache,
            const uint8_t* k_scale, const uint8_t* v_scale, uint16_t* k, uint16_t* v,
            void* stream) {
  if (!cache_shape_ok(heads, dim, pages, page) || tokens < 0 || tokens > kInt32Max ||
      tokens * heads * dim >= kMaxElems)
    return BITDELTA_ERR_SHAPE;
  if (tokens == 0) return BITDELTA_OK;
  if (!k || !v || !slots || !k_cache || !v_cache || !scales_ok(k_scale, v_scale, bits))
    return BITDELTA_ERR_NULL;
  if (!aligned16(k) || !aligned16(v) || !aligned4(slots) || !aligned16(k_cache) ||
      !aligned16(v_cache) || !aligned16(k_scale) || !aligned16(v_scale))
    return BITDELTA_ERR_ALIGN;
  const size_t rows = (size_t)pages * (size_t)page * (size_t)heads;
  const size_t cbytes = cache_bytes(rows, dim, bits), sbytes = scale_bytes(rows, dim, bits);
  const size_t obytes = (size_t)(tokens * heads * dim) * 2u;
  const void* ins[5] = {k_cache, v_cache, k_scale, v_scale, slots};
  const size_t inn[5] = {cbytes, cbytes, sbytes, sbytes, (size_t)tokens * 4u};
  for (int j = 0; j < 5; ++j)
    if (ins[j] && (overlap(k, obytes, ins[j], inn[j]) || overlap(v, obytes, ins[j], inn[j])))
      return BITDELTA_ERR_OVERLAP;
  if (overlap(k, obytes, v, obytes)) return BITDELTA_ERR_OVERLAP;
  const int dev = check_device();
  if (dev != BITDELTA_OK) return dev;
  bd::KvArgs a{};
  a.dst[0] = k;
  a.dst[1] = v;
  a.cache[0] = const_cast<void*>(k_cache);
  a.cache[1] = const_cast<void*>(v_cache);
  a.scale[0] = const_cast<uint8_t*>(k_scale);
  a.scale[1] = const_cast<uint8_t*>(v_scale);
  a.slots = slots;
  a.tokens = tokens;
  a.n_slots = pages * page;
  a.heads = (int)heads;
  a.dim = (int)dim;
  a.page = (int)page;
  a.bits = bits;
  return status_of(bd::launch_kv_read(a, static_cast<hipStream_t>(stream)));
}

bool table_shape_ok(int64_t length, int64_t rot, int64_t dim) {
  return length >= 1 && length <= kInt32Max && rot >= 2 && rot % 2 == 0 && rot <= dim &&
         length * rot < kMaxElems;
}

}  // namespace

BD_EXPORT int bitdelta_rms_norm_block(const uint16_t* x, int64_t x_stride, const uint16_t* post,
                                      const uint16_t* gate, int64_t g_stride, float alpha,
                                      const uint16_t* residual, int64_t r_stride,
                                      const uint16_t* w, float eps, int64_t rows, int64_t cols,
                                      uint16_t* h_out, uint16_t* y, void* stream) {
  if (rows < 0 || rows > kInt32Max || cols < 1 || cols > kMaxDin || rows * cols >= kMaxElems ||
      !std::isfinite(alpha))
    return BITDELTA_ERR_SHAPE;
  if (rows == 0) return BITDELTA_OK;
  if (!x || !residual || !w || !h_out || !y) return BITDELTA_ERR_NULL;
  if (!strides_ok(x_stride, r_stride) || (gate && !strides_ok(g_stride, 0)))
    return BITDELTA_ERR_SHAPE;
  if (!aligned2(x) || !aligned2(post) || !aligned2(gate) || !aligned2(residual) || !aligned2(w) ||
      !aligned2(h_out) || !aligned2(y))
    return BITDELTA_ERR_ALIGN;
  const size_t n = (size_t)rows * (size_t)cols * 2u, one = (size_t)cols * 2u;
  const void* outs[2] = {y, h_out};
  const void* ins[5] = {x, residual, gate, post, w};
  const size_t inn[5] = {span(rows, x_stride, 1, 0, cols), span(rows, r_stride, 1, 0, cols),
                         span(rows, g_stride, 1, 0, cols), one, one};
  for (const void* o : outs)
    for (int j = 0; j < 5; ++j)
      if (ins[j] && overlap(o, n, ins[j], inn[j])) return BITDELTA_ERR_OVERLAP;
  if (overlap(y, n, h_out, n)) return BITDELTA_ERR_OVERLAP;
  const int dev = check_device();
  if (dev != BITDELTA_OK) return dev;
  bd::BlockNormArgs a{};
  a.x = x;
  a.residual = residual;
  a.gate = gate;
  a.post = post;
  a.w = w;
  a.h = h_out;
  a.y = y;
  a.x_stride = x_stride;
  a.r_stride = r_stride;
  a.g_stride = g_stride;
  a.rows = rows;
  a.cols = (int)cols;
  a.alpha = alpha;
  a.eps = eps;
  return status_of(bd::launch_rms_norm_block(a, static_cast<hipStream_t>(stream)));
}

BD_EXPORT int bitdelta_rotary_table(const double* frequencies, int64_t pairs, int64_t first,
                                    int64_t length, double magnitude, float* table, void* stream) {
  if (pairs < 1 || pairs > 32768 || first < 0 || first > kInt32Max || length < 0 ||
      length > kInt32Max || length * pairs * 2 >= kMaxElems)
    return BITDELTA_ERR_SHAPE;
  if (length == 0) return BITDELTA_OK;
  if (!frequencies || !table) return BITDELTA_ERR_NULL;
  if ((reinterpret_cast<uintptr_t>(frequencies) & 7u) || (reinterpret_cast<uintptr_t>(table) & 7u))
    return BITDELTA_ERR_ALIGN;
  if (overlap(table, (size_t)(length * pairs) * 8u, frequencies, (size_t)pairs * 8u))
    return BITDELTA_ERR_OVERLAP;
  const int dev = check_device();
  if (dev != BITDELTA_OK) return dev;
  return status_of(bd::launch_rotary_table(frequencies, (int)pairs, first, length, magnitude,
                                           table, static_cast<hipStream_t>(stream)));
}

BD_EXPORT int bitdelta_rotary(const uint16_t* x, int64_t x_token_stride, int64_t x_head_stride,
                              const int32_t* positions, const float* table, int64_t length,
                              int64_t rot, int32_t interleaved, int64_t tokens, int64_t heads,
                              int64_t dim, uint16_t* out, int64_t out_token_stride,
                              int64_t out_head_stride, void* stream) {
  if (tokens < 0 || tokens > kInt32Max || heads < 1 || heads > 65536 || dim < 2 || dim > 65536 ||
      tokens * heads * dim >= kMaxElems || !table_shape_ok(length, rot, dim) ||
      !strides_ok(x_token_stride, x_head_stride) ||
      !strides_ok(out_token_stride, out_head_stride))
    return BITDELTA_ERR_SHAPE;
  // rows of out lie apart, tokens outside of heads or the other way round
  const int64_t ts = out_token_stride, hs = out_head_stride;
  if (!((hs >= dim || heads == 1) && (ts >= (heads - 1) * hs + dim || tokens <= 1)) &&
      !((ts >= dim || tokens <= 1) && (hs >= (tokens - 1) * ts + dim || heads == 1)))
    return BITDELTA_ERR_SHAPE;
  if (tokens == 0) return BITDELTA_OK;
  if (!x || !positions || !table || !out) return BITDELTA_ERR_NULL;
  if (!aligned2(x) || !aligned2(out) || !aligned4(positions) || !aligned4(table))
    return BITDELTA_ERR_ALIGN;
  const size_t on = span(tokens, ts, heads, hs, dim);
  const bool same = x == out && (tokens == 1 || x_token_stride == ts) &&
                    (heads == 1 || x_head_stride == hs);
  if ((!same && overlap(out, on, x, span(tokens, x_token_stride, heads, x_head_stride, dim))) ||
      overlap(out, on, positions, (size_t)tokens * 4u) ||
      overlap(out, on, table, (size_t)(length * rot) * 4u))
    return BITDELTA_ERR_OVERLAP;
  const int dev = check_device();
  if (dev != BITDELTA_OK) return dev;
  bd::RotaryArgs a{};
  a.x = x;
  a.out = out;
  a.positions = positions;
  a.table = table;
  a.x_token_stride = x_token_stride;
  a.x_head_stride = x_head_stride;
  a.out_token_stride = ts;
  a.out_head_stride = hs;
  a.tokens = tokens;
  a.length = (int)length;
  a.heads = (int)heads;
  a.dim = (int)dim;
  a.rot = (int)rot;
  a.interleaved = interleaved != 0;
  return status_of(bd::launch_rotary(a, static_cast<hipStream_t>(stream)));
}

BD_EXPORT int bitdelta_kv_append(const uint16_t* q, int64_t q_token_stride, int64_t q_head_stride,
                                 const uint16_t* k, int64_t k_token_stride, int64_t k_head_stride,
                                 const uint16_t* v, int64_t v_token_stride, int64_t v_head_stride,
                                 const int32_t* positions, const float* table, int64_t length,
                                 int64_t rot, int32_t interleaved, const int32_t* slots,
                                 int64_t tokens, int64_t heads, int64_t kv_heads, int64_t dim,
                                 int64_t pages, int64_t page, int32_t bits, void* k_cache,
                                 void* v_cache, uint8_t* k_scale, uint8_t* v_scale,
                                 uint16_t* q_out, void* stream) {
  if ((bits != 16 && bits != 8 && bits != 4) || heads < 1 || heads > 1024 ||
      !strides_ok(q_token_stride, q_head_stride) || !table_shape_ok(length, rot, dim))
    return BITDELTA_ERR_SHAPE;
  const int64_t strides[4] = {k_token_stride, k_head_stride, v_token_stride, v_head_stride};
  bd::KvArgs a{};
  const int st = kv_write_args(k, v, strides, slots, tokens, kv_heads, dim, pages, page, bits,
                               k_cache, v_cache, k_scale, v_scale, a);
  if (st != BITDELTA_OK) return st;
  if (tokens * heads * dim >= kMaxElems) return BITDELTA_ERR_SHAPE;
  if (tokens == 0) return BITDELTA_OK;
  if (!q || !positions || !table || !q_out) return BITDELTA_ERR_NULL;
  if (!aligned2(q) || !aligned4(positions) || !aligned4(table) || !aligned2(q_out))
    return BITDELTA_ERR_ALIGN;
  const size_t rows = (size_t)pages * (size_t)page * (size_t)kv_heads;
  const size_t cbytes = cache_bytes(rows, dim, bits), sbytes = scale_bytes(rows, dim, bits);
  const void* outs[5] = {q_out, k_cache, v_cache, k_scale, v_scale};
  const size_t outn[5] = {(size_t)(tokens * heads * dim) * 2u, cbytes, cbytes, sbytes, sbytes};
  const void* ins[6] = {q, positions, table, k, v, slots};
  const size_t inn[6] = {span(tokens, q_token_stride, heads, q_head_stride, dim),
                         (size_t)tokens * 4u, (size_t)(length * rot) * 4u,
                         span(tokens, k_token_stride, kv_heads, k_head_stride, dim),
                         span(tokens, v_token_stride, kv_heads, v_head_stride, dim),
                         (size_t)tokens * 4u};
  for (int i = 0; i < 5; ++i) {
    if (!outs[i]) continue;
    for (int j = 0; j < 6; ++j)
      if (overlap(outs[i], outn[i], ins[j], inn[j])) return BITDELTA_ERR_OVERLAP;
    if (i > 0 && overlap(q_out, outn[0], outs[i], outn[i])) return BITDELTA_ERR_OVERLAP;
  }
  const int dev = check_device();
  if (dev != BITDELTA_OK) return dev;
  bd::RotaryArgs r{};
  r.x = q;
  r.out = q_out;
  r.positions = positions;
  r.table = table;
  r.x_token_stride = q_token_stride;
  r.x_head_stride = q_head_stride;
  r.out_token_stride = heads * dim;
  r.out_head_stride = dim;
  r.tokens = tokens;
  r.length = (int)length;
  r.heads = (int)heads;
  r.dim = (int)dim;
  r.rot = (int)rot;
  r.interleaved = interleaved != 0;
  return status_of(bd::launch_kv_append(a, r, static_cast<hipStream_t>(stream)));
}

BD_EXPORT int bitdelta_kv_write(const uint16_t* k, const uint16_t* v, int64_t k_token_stride,
                                int64_t k_head_stride, int64_t v_token_stride,
                                int64_t v_head_stride, const int32_t* slots, int64_t tokens,
                                int64_t heads, int64_t dim, int64_t pages, int64_t page,
                                void* k_cache, void* v_cache, uint8_t* k_scale, uint8_t* v_scale,
                                void* stream) {
  const int64_t strides[4] = {k_token_stride, k_head_stride, v_token_stride, v_head_stride};
  return kv_write(k, v, strides, slots, tokens, heads, dim, pages, page, k_scale ? 8 : 16, k_cache,
                  v_cache, k_scale, v_scale, stream);
}

BD_EXPORT int bitdelta_kv_write_4bit(const uint16_t* k, const uint16_t* v, int64_t k_token_stride,
                                     int64_t k_head_stride, int64_t v_token_stride,
                                     int64_t v_head_stride, const int32_t* slots, int64_t tokens,
                                     int64_t heads, int64_t dim, int64_t pages, int64_t page,
                                     void* k_cache, void* v_cache, uint8_t* k_scale,
                                     uint8_t* v_scale, void* stream) {
  const int64_t strides[4] = {k_token_stride, k_head_stride, v_token_stride, v_head_stride};
  return kv_write(k, v, strides, slots, tokens, heads, dim, pages, page, 4, k_cache, v_cache,
                  k_scale, v_scale, stream);
}

BD_EXPORT int bitdelta_kv_read(const int32_t* slots, int64_t tokens, int64_t heads, int64_t dim,
                               int64_t pages, int64_t page, const void* k_cache,
                               const void* v_cache, const uint8_t* k_scale,
                               const uint8_t* v_scale, uint16_t* k, uint16_t* v, void* stream) {
  return kv_read(slots, tokens, heads, dim, pages, page, k_scale ? 8 : 16, k_cache, v_cache,
                 k_scale, v_scale, k, v, stream);
}

BD_EXPORT int bitdelta_kv_read_4bit(const int32_t* slots, int64_t tokens, int64_t heads,
                                    int64_t dim, int64_t pages, int64_t page, const void* k_cache,
                                    const void* v_cache, const uint8_t* k_scale,
                                    const uint8_t* v_scale, uint16_t* k, uint16_t* v,
                                    void* stream) {
  return kv_read(slots, tokens, heads, dim, pages, page, 4, k_cache, v_cache, k_scale, v_scale, k,
                 v, stream);
}

namespace {

bool attention_shape_ok(int64_t tokens, int64_t seqs, int64_t max_q, int64_t heads,
                        int64_t kv_heads, int64_t dim, int64_t width, int64_t page) {
  return cache_shape_ok(kv_heads, dim, 1, page) && heads >= kv_heads && heads <= 1024 &&
         heads % kv_heads == 0 && heads / kv_heads <= 64 && tokens >= 0 &&
         tokens <= (kInt32Max >> 1) / heads && seqs >= 0 && seqs <= 65535 && max_q >= 0 &&
         max_q <= kInt32Max && width >= 0 && width <= (int64_t(1) << 30) / page;
}

bd::AttnArgs attention_sizes(int64_t tokens, int64_t seqs, int64_t max_q, int64_t heads,
                             int64_t kv_heads, int64_t dim, int64_t width, int64_t page) {
  bd::AttnArgs a{};
  a.tokens = (int)tokens;
  a.seqs = (int)seqs;
  a.max_q = (int)(max_q < tokens ? max_q : tokens);
  a.heads = (int)heads;
  a.kv_heads = (int)kv_heads;
  a.group = (int)(heads / kv_heads);
  a.dim = (int)dim;
  a.width = (int)width;
  a.page = (int)page;
  return a;
}

}  // namespace

BD_EXPORT size_t bitdelta_paged_attention_workspace_size(int64_t tokens, int64_t seqs,
                                                         int64_t max_q, int64_t heads,
                                                         int64_t kv_heads, int64_t dim,
                                                         int64_t width, int64_t page) {
  if (!attention_shape_ok(tokens, seqs, max_q, heads, kv_heads, dim, width, page)) return 0;
  if (tokens == 0 || seqs == 0 || max_q == 0) return 0;   // nothing to do
  return bd::paged_attention_workspace(
      attention_sizes(tokens, seqs, max_q, heads, kv_heads, dim, width, page));
}

namespace {

int paged_attention(
    int bits, const uint16_t* q, int64_t q_token_stride, int64_t q_head_stride, const void* k_cache,
    const void* v_cache, const uint8_t* k_scale, const uint8_t* v_scale, const int32_t* table,
    const int32_t* cu_q, const int32_t* kv_len, int64_t tokens, int64_t seqs, int64_t max_q,
    int64_t heads, int64_t kv_heads, int64_t dim, int64_t pages, int64_t page, int64_t width,
    float scale, int64_t window, uint16_t* out, void* workspace, size_t workspace_bytes,
    void* stream) {
  // the running maximum is taken of the unscaled scores: scale must keep their
  // order, and -infinity times it must stay -infinity
  const float scale_log2 = scale * 1.4426950408889634f;
  if (!attention_shape_ok(tokens, seqs, max_q, heads, kv_heads, dim, width, page) ||
      !cache_shape_ok(kv_heads, dim, pages, page) || window < 0 ||
      !(scale_log2 >= 1.17549435e-38f && scale_log2 < INFINITY) || q_token_stride < 0 ||
      q_head_stride < 0 || q_token_stride >= kMaxElems || q_head_stride >= kMaxElems)
    return BITDELTA_ERR_SHAPE;
  if (tokens == 0 || seqs == 0 || max_q == 0) return BITDELTA_OK;
  if (!q || !k_cache || !v_cache || (!table && width > 0) || !cu_q || !kv_len || !out ||
      !scales_ok(k_scale, v_scale, bits))
    return BITDELTA_ERR_NULL;
  if (!aligned2(q) || !aligned16(k_cache) || !aligned16(v_cache) || !aligned16(k_scale) ||
      !aligned16(v_scale) || !aligned4(table) || !aligned4(cu_q) || !aligned4(kv_len) ||
      !aligned16(out) || !aligned16(workspace))
    return BITDELTA_ERR_ALIGN;
  bd::AttnArgs a = attention_sizes(tokens, seqs, max_q, heads, kv_heads, dim, width, page);
  const size_t need = bd::paged_attention_workspace(a);
  if (need > 0 && (!workspace || workspace_bytes < need)) return BITDELTA_ERR_WORKSPACE;
  const size_t rows = (size_t)pages * (size_t)page * (size_t)kv_heads;
  const size_t cbytes = cache_bytes(rows, dim, bits), sbytes = scale_bytes(rows, dim, bits);
  const void* outs[2] = {out, need ? workspace : nullptr};
  const size_t outn[2] = {(size_t)(tokens * heads * dim) * 2u, need};
  const void* ins[8] = {q, k_cache, v_cache, k_scale, v_scale, table, cu_q, kv_len};
  const size_t inn[8] = {span(tokens, q_token_stride, heads, q_head_stride, dim), cbytes, cbytes,
                         sbytes, sbytes, (size_t)(seqs * width) * 4u, (size_t)(seqs + 1) * 4u,
                         (size_t)seqs * 4u};
  for (int i = 0; i < 2; ++i)
    for (int j = 0; j < 8; ++j)
      if (outs[i] && ins[j] && overlap(outs[i], outn[i], ins[j], inn[j]))
        return BITDELTA_ERR_OVERLAP;
  if (outs[1] && overlap(outs[0], outn[0], outs[1], outn[1])) return BITDELTA_ERR_OVERLAP;
  const int dev = check_device();
  if (dev != BITDELTA_OK) return dev;
  a.q = q;
  a.q_token_stride = q_token_stride;
  a.q_head_stride = q_head_stride;
  a.cache[0] = static_cast<const uint8_t*>(k_cache);
  a.cache[1] = static_cast<const uint8_t*>(v_cache);
  a.scale[0] = k_scale;
  a.scale[1] = v_scale;
  a.table = table;
  a.cu_q = cu_q;
  a.kv_len = kv_len;
  a.pages = pages;
  a.bits = bits;
  // a window that no sequence can fill hides nothing; what is left keeps
  // positions minus the window inside an int
  a.window = (int)(window < width * page ? window : 0);
  a.scale_log2 = scale_log2;
  a.out = out;
  a.partial = static_cast<float*>(workspace);
  return status_of(bd::launch_paged_attention(a, static_cast<hipStream_t>(stream)));
}

}  // namespace

BD_EXPORT int bitdelta_paged_attention(
    const uint16_t* q, int64_t q_token_stride, int64_t q_head_stride, const void* k_cache,
    const void* v_cache, const uint8_t* k_scale, const uint8_t* v_scale, const int32_t* table,
    const int32_t* cu_q, const int32_t* kv_len, int64_t tokens, int64_t seqs, int64_t max_q,
    int64_t heads, int64_t kv_heads, int64_t dim, int64_t pages, int64_t page, int64_t width,
    float scale, int64_t window, uint16_t* out, void* workspace, size_t workspace_bytes,
    void* stream) {
  return paged_attention(k_scale ? 8 : 16, q, q_token_stride, q_head_stride, k_cache, v_cache,
                         k_scale, v_scale, table, cu_q, kv_len, tokens, seqs, max_q, heads,
                         kv_heads, dim, pages, page, width, scale, window, out, workspace,
                         workspace_bytes, stream);
}

BD_EXPORT int bitdelta_paged_attention_4bit(
    const uint16_t* q, int64_t q_token_stride, int64_t q_head_stride, const void* k_cache,
    const void* v_cache, const uint8_t* k_scale, const uint8_t* v_scale, const int32_t* table,
    const int32_t* cu_q, const int32_t* kv_len, int64_t tokens, int64_t seqs, int64_t max_q,
    int64_t heads, int64_t kv_heads, int64_t dim, int64_t pages, int64_t page, int64_t width,
    float scale, int64_t window, uint16_t* out, void* workspace, size_t workspace_bytes,
    void* stream) {
  return paged_attention(4, q, q_token_stride, q_head_stride, k_cache, v_cache, k_scale, v_scale,
                         table, cu_q, kv_len, tokens, seqs, max_q, heads, kv_heads, dim, pages,
                         page, width, scale, window, out, workspace, workspace_bytes, stream);
}

BD_EXPORT int bitdelta_probe_stream_read(const void* src, size_t bytes, int32_t workgroups,
                                         uint32_t* sink, void* stream) {
  if (!src || !sink) return BITDELTA_ERR_NULL;
  if (bytes == 0 || bytes % 16 != 0 || workgroups < 1 || workgroups > (1 << 20))
    return BITDELTA_ERR_SHAPE;
  if (!aligned16(src) || (reinterpret_cast<uintptr_t>(sink) & 3u)) return BITDELTA_ERR_ALIGN;
  if (overlap(sink, 1024, src, bytes)) return BITDELTA_ERR_OVERLAP;
  const int dev = check_device();
  if (dev != BITDELTA_OK) return dev;
  return status_of(bd::launch_probe_read(src, bytes, workgroups, sink,
                                         static_cast<hipStream_t>(stream)));
}

BD_EXPORT int bitdelta_probe_decode_loads(const void* w, const void* signs, const void* x,
                                          int32_t mode, uint32_t* sink, void* stream) {
  if (!w || !signs || !x || !sink) return BITDELTA_ERR_NULL;
  if (mode < 0 || mode > 5) return BITDELTA_ERR_MODE;
  if (!aligned16(w) || !aligned16(x) || (reinterpret_cast<uintptr_t>(signs) & 3u) ||
      (reinterpret_cast<uintptr_t>(sink) & 3u))
    return BITDELTA_ERR_ALIGN;
  if (overlap(sink, 1024, w, size_t(4096) * 8192) || overlap(sink, 1024, signs, size_t(1) << 21) ||
      overlap(sink, 1024, x, 8192))
    return BITDELTA_ERR_OVERLAP;
  const int dev = check_device();
  if (dev != BITDELTA_OK) return dev;
  return status_of(bd::launch_probe_decode_loads(w, signs, x, mode, sink,
                                                 static_cast<hipStream_t>(stream)));
}

BD_EXPORT int bitdelta_probe_mfma_bf16(int32_t workgroups, int32_t iters, float* sink,
                                       void* stream) {
  if (!sink) return BITDELTA_ERR_NULL;
  if (workgroups < 1 || workgroups > (1 << 20) || iters < 1 || iters > (1 << 24))
    return BITDELTA_ERR_SHAPE;
  if (reinterpret_cast<uintptr_t>(sink) & 3u) return BITDELTA_ERR_ALIGN;
  const int dev = check_device();
  if (dev != BITDELTA_OK) return dev;
  return status_of(bd::launch_probe_mfma(workgroups, iters, sink,
                                         static_cast<hipStream_t>(stream)));
}
