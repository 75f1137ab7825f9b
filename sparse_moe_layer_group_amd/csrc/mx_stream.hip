// Products of microscaled operands, tokens by 4-bit weights, straight from
// memory to registers.
//
//   out[t][n] = residual + act(sum_k x[t][k] w[n][k] + bias[n])
//   dual: mid[t][n] = act(x w^T) * (x w2^T)
//
// A workgroup of eight waves takes 16 weight rows (dual: 8 of each matrix, the
// same columns) and up to 64 tokens; the waves take the contraction's steps of
// 128 in eight ranges and their sums are joined through LDS in wave order.
// One v_mfma_scale_f32_16x16x128_f8f6f4 is a step of 16 weight rows and 16
// tokens with the blocks' scales.  Lane l of 4-bit codes has row l % 16, block
// l / 16 of the step (16 bytes); of 8-bit codes the 16-byte chunks l / 16 and
// l / 16 + 4 of its row's 128; its scale is block l / 16's.
#include "mx.h"

namespace moe {

namespace {

constexpr int kWaves = 8;  // of a workgroup
constexpr int kRows = 16;  // weight rows of a workgroup

}  // namespace

template <int FORM, int TT, bool DUAL, bool EXACT> __global__ __launch_bounds__(64 * kWaves) void mx_stream_kernel(MxArgs g) {
  constexpr int NC = DUAL ? kRows / 2 : kRows, XB = mx_step_bytes(FORM);
  __shared__ float sums[kWaves][TT * 16][kRows + 1];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int nt = (g.N + NC - 1) / NC;
  const int n0 = int(blockIdx.x % nt) * NC;
  const int64_t t0 = int64_t(blockIdx.x / nt) * (16 * TT);
  const int r = lane & 15, q = lane >> 4;
  // this lane's weight row and token rows; rows past the end repeat the last
  const int64_t n = min(n0 + (DUAL ? r & 7 : r), g.N - 1);
  const uint8_t* w = (DUAL && r >= 8 ? g.w2 : g.w) + n * g.steps * 64 + 16 * q;
  const uint8_t* sw = (DUAL && r >= 8 ? g.sw2 : g.sw) + n * g.steps * 4 + q;
  const uint8_t *x[TT], *sx[TT];
#pragma unroll
  for (int i = 0; i < TT; ++i) {
    const int64_t t = min(t0 + 16 * i + r, g.T - 1);
    x[i] = g.x + t * g.steps * XB + 16 * q;
    sx[i] = g.sx + t * g.steps * 4 + q;
  }
  f32x4 acc[TT];
#pragma unroll
  for (int i = 0; i < TT; ++i) acc[i] = f32x4{0.f, 0.f, 0.f, 0.f};
  const int s1 = g.steps * (wave + 1) / kWaves;
  for (int s = g.steps * wave / kWaves; s < s1; ++s) {
    const i32x4 a = *reinterpret_cast<const i32x4*>(w + s * 64);
    const int swa = sw[s * 4];
#pragma unroll
    for (int i = 0; i < TT; ++i) {
      const i32x4 lo = *reinterpret_cast<const i32x4*>(x[i] + s * XB);
      i32x4 hi = {0, 0, 0, 0};
      if (FORM == kMxE4M3) hi = *reinterpret_cast<const i32x4*>(x[i] + s * XB + 64);
      acc[i] = mx_multiply<FORM, EXACT>(a, swa, lo, hi, int(sx[i][s * 4]), acc[i]);
    }
  }
  // accumulator v of lane l: weight row 4 (l / 16) + v, token l % 16
#pragma unroll
  for (int i = 0; i < TT; ++i)
#pragma unroll
    for (int v = 0; v < 4; ++v) sums[wave][16 * i + r][4 * q + v] = acc[i][v];
  __syncthreads();
  for (int id = threadIdx.x; id < TT * 16 * NC; id += 64 * kWaves) {
    const int row = id / NC, c = id % NC, col = n0 + c;
    const int64_t t = t0 + row;
    if (t >= g.T || col >= g.N) continue;
    float v = 0.f, u = 0.f;
#pragma unroll
    for (int k = 0; k < kWaves; ++k) {
      v += sums[k][row][c];
      if (DUAL) u += sums[k][row][kRows / 2 + c];
    }
    if (DUAL) {
      g.mid[t * g.ld_out + col] = act_one(g.act, v) * u;
      continue;
    }
    if (g.bias) v += g.f32 ? static_cast<const float*>(g.bias)[col] : bf16_to_f32(static_cast<const bf16_t*>(g.bias)[col]);
    v = act_one(g.act, v);
    if (g.residual) {
      const int64_t at = t * g.ld_residual + col;
      v += g.f32 ? static_cast<const float*>(g.residual)[at] : bf16_to_f32(static_cast<const bf16_t*>(g.residual)[at]);
    }
    if (g.f32) static_cast<float*>(g.out)[t * g.ld_out + col] = v;
    else static_cast<bf16_t*>(g.out)[t * g.ld_out + col] = f32_to_bf16(v);
  }
}

namespace {

template <int FORM, int TT, bool EXACT> hipError_t launch_tokens(const MxArgs& g, hipStream_t st) {
  const int64_t nc = g.w2 ? kRows / 2 : kRows;
  const int64_t grid = (g.N + nc - 1) / nc * ((g.T + 16 * TT - 1) / (16 * TT));
  if (grid > 0x7fffffff) return hipErrorInvalidValue;
  if (g.w2)
    hipLaunchKernelGGL((mx_stream_kernel<FORM, TT, true, EXACT>), dim3(unsigned(grid)), dim3(64 * kWaves), 0, st, g);
  else
    hipLaunchKernelGGL((mx_stream_kernel<FORM, TT, false, EXACT>), dim3(unsigned(grid)), dim3(64 * kWaves), 0, st, g);
  return hipGetLastError();
}
template <int FORM, bool EXACT> hipError_t launch_form(const MxArgs& g, hipStream_t st) {
  if (g.T <= 16) return launch_tokens<FORM, 1, EXACT>(g, st);
  if (g.T <= 32) return launch_tokens<FORM, 2, EXACT>(g, st);
  return launch_tokens<FORM, 4, EXACT>(g, st);
}

}  // namespace

hipError_t launch_mx_stream(const MxArgs& g, int form, hipStream_t st) {
  if (g.T < 1 || g.N < 1 || g.steps < 1) return hipErrorInvalidValue;
  if (form == kMxE2M1) return launch_form<kMxE2M1, false>(g, st);
  return g.exact ? launch_form<kMxE4M3, true>(g, st) : launch_form<kMxE4M3, false>(g, st);
}

}  // namespace moe
