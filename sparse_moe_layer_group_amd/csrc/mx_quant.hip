// Matrices to microscaled form and back.
//
//   e = max(floor(log2 max |v|) - emax, -127) over a block of 32, code = v 2^-e
//   rounded to nearest even and saturated; back: code 2^e
//
// Memory-bound: an element's bytes in, one or a half out.  A lane has 8
// consecutive elements (one or two 16-byte loads), a quad of lanes a block, so
// the largest magnitude takes two lane moves; a workgroup's lanes lie along a row
// as far as it goes, then over rows.
#include <algorithm>

#include "mx.h"

namespace moe {

namespace {

constexpr int kLanes = 256;

// lane columns of a workgroup (a power of two of at least 16): 8 elements each
int lane_columns(int cols) {
  const int need = int(mx_steps(cols)) * 16;
  int n = 16;
  while (n < need && n < kLanes) n *= 2;
  return n;
}

}  // namespace

template <typename TE, int FORM>
__global__ __launch_bounds__(kLanes) void mx_quantize_kernel(const TE* x, int64_t ld, int64_t rows, int cols, int lx,
                                                             uint8_t* codes, uint8_t* scales) {
  const int pieces = (cols + 127) / 128 * 16;  // of a padded row
  const int across = (pieces + lx - 1) / lx;
  const int64_t row = int64_t(blockIdx.x / across) * (kLanes / lx) + threadIdx.x / lx;
  const int piece = int(blockIdx.x % across) * lx + threadIdx.x % lx;
  if (row >= rows || piece >= pieces) return;  // whole steps of 16 lanes
  float v[8];
  load8<false>(x + row * ld, piece * 8, cols, v);
  const uint32_t byte = mx_quad_scale<FORM>(v);
  constexpr int W = MxForm<FORM>::WORDS;
  uint32_t o[W];
  mx_encode8<FORM>(v, byte, o);
  uint32_t* to = reinterpret_cast<uint32_t*>(codes) + (row * pieces + piece) * W;
#pragma unroll
  for (int i = 0; i < W; ++i) to[i] = o[i];
  if ((piece & 3) == 0) scales[(row * pieces + piece) / 4] = uint8_t(byte);
}

template <typename TE, int FORM>
__global__ __launch_bounds__(kLanes) void mx_dequantize_kernel(const uint8_t* codes, const uint8_t* scales, int64_t rows,
                                                               int cols, int lx, TE* y, int64_t ld) {
  const int pieces = (cols + 127) / 128 * 16;
  const int across = (pieces + lx - 1) / lx;
  const int64_t row = int64_t(blockIdx.x / across) * (kLanes / lx) + threadIdx.x / lx;
  const int piece = int(blockIdx.x % across) * lx + threadIdx.x % lx;
  if (row >= rows || piece * 8 >= cols) return;
  const float scale = mx_power(scales[(row * pieces + piece) / 4]);
  constexpr int W = MxForm<FORM>::WORDS;
  const uint32_t* from = reinterpret_cast<const uint32_t*>(codes) + (row * pieces + piece) * W;
  float v[8];
  if constexpr (FORM == kMxE4M3) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const auto lo = __builtin_amdgcn_cvt_pk_f32_fp8(int(from[h]), false);
      const auto hi = __builtin_amdgcn_cvt_pk_f32_fp8(int(from[h]), true);
      v[4 * h] = lo[0], v[4 * h + 1] = lo[1], v[4 * h + 2] = hi[0], v[4 * h + 3] = hi[1];
    }
  } else {
    const uint32_t c = from[0];
    const auto a = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, 1.0f, 0);
    const auto b = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, 1.0f, 1);
    const auto d = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, 1.0f, 2);
    const auto e = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, 1.0f, 3);
    v[0] = a[0], v[1] = a[1], v[2] = b[0], v[3] = b[1], v[4] = d[0], v[5] = d[1], v[6] = e[0], v[7] = e[1];
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] *= scale;
  store8<false>(y + row * ld, piece * 8, cols, v);
}

namespace {

// Rows of a launch: a grid has less than 2^32 threads.
constexpr int64_t kMostGroups = int64_t(1) << 23;
template <class F> hipError_t by_rows(int64_t rows, int cols, F launch) {
  const int lx = lane_columns(cols), down = kLanes / lx;
  const int64_t across = (mx_steps(cols) * 16 + lx - 1) / lx, most = kMostGroups / across * down;
  for (int64_t first = 0; first < rows; first += most) {
    const int64_t n = std::min(most, rows - first);
    launch(first, n, lx, dim3(unsigned(across * ((n + down - 1) / down))));
    const hipError_t err = hipGetLastError();
    if (err != hipSuccess) return err;
  }
  return hipSuccess;
}
template <typename TE, int FORM> hipError_t quantize(const void* x, int64_t ld, int64_t rows, int cols, uint8_t* codes,
                                                     uint8_t* scales, hipStream_t st) {
  const int64_t steps = mx_steps(cols);
  return by_rows(rows, cols, [&](int64_t first, int64_t n, int lx, dim3 grid) {
    hipLaunchKernelGGL((mx_quantize_kernel<TE, FORM>), grid, dim3(kLanes), 0, st, static_cast<const TE*>(x) + first * ld,
                       ld, n, cols, lx, codes + first * steps * mx_step_bytes(FORM), scales + first * steps * 4);
  });
}
template <typename TE, int FORM> hipError_t dequantize(const uint8_t* codes, const uint8_t* scales, int64_t rows,
                                                       int cols, void* y, int64_t ld, hipStream_t st) {
  const int64_t steps = mx_steps(cols);
  return by_rows(rows, cols, [&](int64_t first, int64_t n, int lx, dim3 grid) {
    hipLaunchKernelGGL((mx_dequantize_kernel<TE, FORM>), grid, dim3(kLanes), 0, st,
                       codes + first * steps * mx_step_bytes(FORM), scales + first * steps * 4, n, cols, lx,
                       static_cast<TE*>(y) + first * ld, ld);
  });
}

}  // namespace

hipError_t launch_mx_quantize(int form, bool f32, const void* x, int64_t ld, int64_t rows, int cols, uint8_t* codes,
                              uint8_t* scales, hipStream_t st) {
  if (form == kMxE4M3)
    return f32 ? quantize<float, kMxE4M3>(x, ld, rows, cols, codes, scales, st)
               : quantize<bf16_t, kMxE4M3>(x, ld, rows, cols, codes, scales, st);
  return f32 ? quantize<float, kMxE2M1>(x, ld, rows, cols, codes, scales, st)
             : quantize<bf16_t, kMxE2M1>(x, ld, rows, cols, codes, scales, st);
}
hipError_t launch_mx_dequantize(int form, bool f32, const uint8_t* codes, const uint8_t* scales, int64_t rows, int cols,
                                void* y, int64_t ld, hipStream_t st) {
  if (form == kMxE4M3)
    return f32 ? dequantize<float, kMxE4M3>(codes, scales, rows, cols, y, ld, st)
               : dequantize<bf16_t, kMxE4M3>(codes, scales, rows, cols, y, ld, st);
  return f32 ? dequantize<float, kMxE2M1>(codes, scales, rows, cols, y, ld, st)
             : dequantize<bf16_t, kMxE2M1>(codes, scales, rows, cols, y, ld, st);
}

}  // namespace moe
