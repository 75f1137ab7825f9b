// Matrices to microscaled form and back.
//
//   e = max(floor(log2 max |v|) - emax, -127) over a block of 32, code = v 2^-e
//   rounded to nearest even and saturated; back: code 2^e
//
// Memory-bound: an element's bytes in, one or a half out.  A lane has 8
// consecutive elements (one or two 16-byte loads), a quad of lanes a block, so
// the largest magnitude takes two lane moves.  Pieces of 8 are dealt to lanes in a
// row, rows one after the other whatever their length, two to a lane with both
// loads in flight (one: 8192 x 7168 to 4 bits 34.5 us, two 32.5, four 35.6; with
// rows given whole powers of two of lanes 32.5, as here 28.9, and 50000 rows of 520
// to 8 bits 23.7 and 18.3).
//
// Measured, a call: 8192 x 7168 in bfloat16 to 8 bits 34.1 us (178 MB at 5.2 TB/s, the
// rate of a large copy) and back 32.2, to 4 bits 28.9 (147 MB, 5.1 TB/s) and back 30.1;
// 777 x 1001 in float32 3 us, a launch's latency.
#include <algorithm>

#include "mx.h"

namespace moe {

namespace {

constexpr int kLanes = 256;
constexpr int kPieces = 2;  // of a lane, kLanes apart

// Elements 8 c .. 8 c + 7 of a row of whole steps: one of `all` pieces, row after row.
struct Piece {
  int64_t row;
  int c;
  bool in;
};
MOE_DEV Piece piece_of(int k, uint32_t all, uint32_t pieces) {
  const uint32_t id = (blockIdx.x * kPieces + k) * kLanes + threadIdx.x, row = id / pieces;
  return Piece{row, int(id - row * pieces), id < all};
}

}  // namespace

template <typename TE, int FORM>
__global__ __launch_bounds__(kLanes) void mx_quantize_kernel(const TE* x, int64_t ld, uint32_t all, int cols,
                                                             uint8_t* codes, uint8_t* scales) {
  const uint32_t pieces = (cols + 127) / 128 * 16;  // of a padded row
  float v[kPieces][8];
  Piece p[kPieces];
#pragma unroll
  for (int k = 0; k < kPieces; ++k) {
    p[k] = piece_of(k, all, pieces);
    if (p[k].in) load8<false>(x + p[k].row * ld, p[k].c * 8, cols, v[k]);
  }
#pragma unroll
  for (int k = 0; k < kPieces; ++k) {
    if (!p[k].in) break;  // whole steps of 16 lanes
    const uint32_t byte = mx_quad_scale<FORM>(v[k]);
    constexpr int W = MxForm<FORM>::WORDS;
    uint32_t o[W];
    mx_encode8<FORM>(v[k], byte, o);
    const int64_t at = p[k].row * pieces + p[k].c;
    uint32_t* to = reinterpret_cast<uint32_t*>(codes) + at * W;
    if constexpr (W == 2) *reinterpret_cast<uint2*>(to) = uint2{o[0], o[1]};
    else *to = o[0];
    if ((p[k].c & 3) == 0) scales[at / 4] = uint8_t(byte);
  }
}

template <int FORM> MOE_DEV void decode8(const uint32_t* from, float (&v)[8]) {
  if constexpr (FORM == kMxE4M3) {
    const uint2 c = *reinterpret_cast<const uint2*>(from);
    const auto a = __builtin_amdgcn_cvt_pk_f32_fp8(int(c.x), false), b = __builtin_amdgcn_cvt_pk_f32_fp8(int(c.x), true);
    const auto d = __builtin_amdgcn_cvt_pk_f32_fp8(int(c.y), false), e = __builtin_amdgcn_cvt_pk_f32_fp8(int(c.y), true);
    v[0] = a[0], v[1] = a[1], v[2] = b[0], v[3] = b[1], v[4] = d[0], v[5] = d[1], v[6] = e[0], v[7] = e[1];
  } else {
    const uint32_t c = from[0];
    const auto a = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, 1.0f, 0);
    const auto b = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, 1.0f, 1);
    const auto d = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, 1.0f, 2);
    const auto e = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, 1.0f, 3);
    v[0] = a[0], v[1] = a[1], v[2] = b[0], v[3] = b[1], v[4] = d[0], v[5] = d[1], v[6] = e[0], v[7] = e[1];
  }
}

template <typename TE, int FORM>
__global__ __launch_bounds__(kLanes) void mx_dequantize_kernel(const uint8_t* codes, const uint8_t* scales, uint32_t all,
                                                               int cols, TE* y, int64_t ld) {
  const uint32_t pieces = (cols + 127) / 128 * 16;
  float v[kPieces][8], scale[kPieces];
  Piece p[kPieces];
#pragma unroll
  for (int k = 0; k < kPieces; ++k) {
    p[k] = piece_of(k, all, pieces);
    p[k].in = p[k].in && p[k].c * 8 < cols;
    if (p[k].in) {
      const int64_t at = p[k].row * pieces + p[k].c;
      scale[k] = mx_power(scales[at / 4]);
      decode8<FORM>(reinterpret_cast<const uint32_t*>(codes) + at * MxForm<FORM>::WORDS, v[k]);
    }
  }
#pragma unroll
  for (int k = 0; k < kPieces; ++k) {
    if (!p[k].in) continue;
#pragma unroll
    for (int i = 0; i < 8; ++i) v[k][i] *= scale[k];
    store8<false>(y + p[k].row * ld, p[k].c * 8, cols, v[k]);
  }
}

namespace {

// Rows of a launch: a grid has less than 2^32 threads, and pieces are counted in 32 bits.
template <class F> hipError_t by_rows(int64_t rows, int cols, F launch) {
  const int64_t pieces = mx_steps(cols) * 16, most = (int64_t(1) << 30) / pieces;
  for (int64_t first = 0; first < rows; first += most) {
    const int64_t all = std::min(most, rows - first) * pieces;
    launch(first, uint32_t(all), dim3(unsigned((all + kPieces * kLanes - 1) / (kPieces * kLanes))));
    const hipError_t err = hipGetLastError();
    if (err != hipSuccess) return err;
  }
  return hipSuccess;
}
template <typename TE, int FORM> hipError_t quantize(const void* x, int64_t ld, int64_t rows, int cols, uint8_t* codes,
                                                     uint8_t* scales, hipStream_t st) {
  const int64_t steps = mx_steps(cols);
  return by_rows(rows, cols, [&](int64_t first, uint32_t all, dim3 grid) {
    hipLaunchKernelGGL((mx_quantize_kernel<TE, FORM>), grid, dim3(kLanes), 0, st, static_cast<const TE*>(x) + first * ld,
                       ld, all, cols, codes + first * steps * mx_step_bytes(FORM), scales + first * steps * 4);
  });
}
template <typename TE, int FORM> hipError_t dequantize(const uint8_t* codes, const uint8_t* scales, int64_t rows,
                                                       int cols, void* y, int64_t ld, hipStream_t st) {
  const int64_t steps = mx_steps(cols);
  return by_rows(rows, cols, [&](int64_t first, uint32_t all, dim3 grid) {
    hipLaunchKernelGGL((mx_dequantize_kernel<TE, FORM>), grid, dim3(kLanes), 0, st,
                       codes + first * steps * mx_step_bytes(FORM), scales + first * steps * 4, all, cols,
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
