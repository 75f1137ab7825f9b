// Products of microscaled operands for few tokens (a serving step): the 4-bit
// weights pass through once, from memory to registers, and are all that counts.
//
//   out[t][n] = residual + act(sum_k x[t][k] w[n][k] + bias[n])
//   dual: act(x w^T) * (x w2^T), in float32
//
// One v_mfma_scale_f32_16x16x128_f8f6f4 takes a step of 128 of 16 weight rows and
// 16 tokens with the blocks' scales.  Lane l of 4-bit codes has row l % 16, block
// l / 16 of the step (16 bytes); of 8-bit codes the 16-byte chunks l / 16 and
// l / 16 + 4 of its row's 128; its scale is block l / 16's.
//
// Memory-bound, so what matters is that enough bytes are in flight on every CU: one
// alone has about 35 KB of loads under way, 20 GB/s of what comes from memory.  So
// a workgroup takes no more than 16 weight rows (dual: 8 of each matrix, the same
// columns), with eight waves, each a range of the contraction with the loads of its
// next four steps in flight during four.  Their sums are joined through LDS in wave
// order.  The dual product cannot be quantised here, as its blocks are four
// workgroups': it stays in float32, and the product that reads it quantises what
// it reads, in every workgroup again, to the codes that mx_quant.hip would write.
// (32 columns a workgroup, which quantises them: 64 workgroups for a block of hidden
// 7168 and inter 2048, one token, 13 to 16 us.)
//
// Measured, one token of 8 bits: 7168 -> 7168 8.9 us (27 MB of weights, 3.1 TB/s, which
// counts 3 us of a launch), gate and up of 7168 -> 2048 6.0 (15.6 MB), down from there
// with the middle's quantising 7.0 (7.8 MB).  An instruction is full at 16 tokens, so
// that is the most: calls of 16 here and 17 by tiles, 7168 -> 7168 12.7 and 12.0 us (4
// bits 9.7 and 13.4), 7168 -> 2048 8.2 and 11.0, the block of these 19.2 and 19.0.
#include "dense_tiles.h"
#include "mx.h"

namespace moe {

namespace {

constexpr int kWaves = 8;  // of a workgroup
constexpr int kRows = 16;  // weight rows of a workgroup
constexpr int kSteps = 4;  // of the loads in flight

// MIDDLE: x is float32
template <int FORM_, bool DUAL_, bool EXACT_, bool MIDDLE_> struct MxStreamShape {
  static constexpr int FORM = FORM_;
  static constexpr bool DUAL = DUAL_, EXACT = EXACT_, MIDDLE = MIDDLE_;
};

// 16 values as codes (8 bits: four words; 4 bits: two)
template <int FORM> MOE_DEV void encode16(const float (&v)[16], uint32_t byte, uint32_t (&o)[2 * MxForm<FORM>::WORDS]) {
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    float a[8];
    uint32_t w[MxForm<FORM>::WORDS];
#pragma unroll
    for (int i = 0; i < 8; ++i) a[i] = v[8 * h + i];
    mx_encode8<FORM>(a, byte, w);
#pragma unroll
    for (int i = 0; i < MxForm<FORM>::WORDS; ++i) o[MxForm<FORM>::WORDS * h + i] = w[i];
  }
}
MOE_DEV uint32_t load16(const float* p, float (&v)[16]) {  // and their largest magnitude
  uint32_t m = 0;
#pragma unroll
  for (int h = 0; h < 4; ++h) {
    const f32x4 a = reinterpret_cast<const f32x4*>(p)[h];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[4 * h + i] = a[i];
      m = max(m, magnitude(a[i]));
    }
  }
  return m;
}
// A step of a float32 row as operand and scale; p: the row's values of the step.
// 4 bits: a lane has block q.  8 bits: chunk q, half of block q / 2, and chunk q + 4,
// half of block 2 + q / 2; the other halves are lane ^ 16's, and block q's scale is
// with lane 2 (q & 1) of the row, its first or (q >= 2) its second.
template <int FORM> MOE_DEV void quantise_step(const float* p, int q, int lane, i32x4& lo, i32x4& hi, int& scale) {
  float a[16], b[16];
  if constexpr (FORM == kMxE2M1) {
    uint32_t m = load16(p + 32 * q, a);
    m = max(m, load16(p + 32 * q + 16, b));
    const uint32_t byte = mx_scale_byte<FORM>(m);
    uint32_t oa[2], ob[2];
    encode16<FORM>(a, byte, oa);
    encode16<FORM>(b, byte, ob);
    lo = i32x4{int(oa[0]), int(oa[1]), int(ob[0]), int(ob[1])};
    scale = int(byte);
  } else {
    uint32_t ma = load16(p + 16 * q, a), mb = load16(p + 64 + 16 * q, b);
    ma = max(ma, uint32_t(__shfl_xor(int(ma), 16, 64)));
    mb = max(mb, uint32_t(__shfl_xor(int(mb), 16, 64)));
    const uint32_t ba = mx_scale_byte<FORM>(ma), bb = mx_scale_byte<FORM>(mb);
    uint32_t oa[4], ob[4];
    encode16<FORM>(a, ba, oa);
    encode16<FORM>(b, bb, ob);
    lo = i32x4{int(oa[0]), int(oa[1]), int(oa[2]), int(oa[3])};
    hi = i32x4{int(ob[0]), int(ob[1]), int(ob[2]), int(ob[3])};
    const int two = __shfl(int(ba | bb << 8), (lane & 15) + 32 * (q & 1), 64);
    scale = q < 2 ? two & 255 : two >> 8;
  }
}

// what a wave needs of kSteps steps: of the weights, and of the tokens
struct WeightSteps {
  i32x4 w[kSteps];
  u32x4 s;
};
struct TokenSteps {
  i32x4 lo[kSteps], hi[kSteps];
  u32x4 s;
};

}  // namespace

template <class S> __global__ __launch_bounds__(64 * kWaves) void mx_stream_kernel(MxArgs g) {
  constexpr int NC = S::DUAL ? kRows / 2 : kRows, XB = mx_step_bytes(S::FORM);
  __shared__ float sums[kWaves][kRows][17];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int n0 = blockIdx.x * NC;
  const int r = lane & 15, q = lane >> 4;
  // this lane's weight row and token row; rows past the end repeat the last
  const bool second = S::DUAL && r >= 8;
  const int n = min(n0 + (S::DUAL ? r & 7 : r), g.N - 1);
  const int t = min(r, int(g.T) - 1);
  const uint8_t* w = (second ? g.w2 : g.w) + int64_t(n) * g.steps * 64 + 16 * q;
  const uint8_t* x = S::MIDDLE ? nullptr : g.x + int64_t(t) * g.steps * XB + 16 * q;
  // Scales as buffers (below 2^32 bytes): those of four steps are one load, wherever
  // the matrix ends.  (dual: each lane's of one matrix, nothing of the other)
  constexpr int kNowhere = int(0xfffffff0u);
  const __amdgpu_buffer_rsrc_t rsw = buffer_rsrc(g.sw, uint32_t(g.N) * g.steps * 4u);
  const __amdgpu_buffer_rsrc_t rsw2 = buffer_rsrc(S::DUAL ? g.sw2 : g.sw, uint32_t(g.N) * g.steps * 4u);
  const __amdgpu_buffer_rsrc_t rsx = buffer_rsrc(g.sx, S::MIDDLE ? 0u : uint32_t(g.T) * g.steps * 4u);
  const float* middle = S::MIDDLE ? g.middle + int64_t(t) * g.steps * 128 : nullptr;
  const int s0 = g.steps * wave / kWaves, s1 = g.steps * (wave + 1) / kWaves;

  auto scales = [](__amdgpu_buffer_rsrc_t rs, int at) {
    return __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(rs, at, 0, 0));
  };
  auto load_weights = [&](WeightSteps& f, int s) {
    const int at = (n * g.steps + s) * 4;
    f.s = scales(rsw, second ? kNowhere : at);
    if (S::DUAL) f.s |= scales(rsw2, second ? at : kNowhere);
#pragma unroll
    for (int k = 0; k < kSteps; ++k) {
      f.w[k] = i32x4{0, 0, 0, 0};
      if (s + k < s1) f.w[k] = *reinterpret_cast<const i32x4*>(w + int64_t(s + k) * 64);
    }
  };
  auto load_tokens = [&](TokenSteps& f, int s) {
    f.s = scales(rsx, (t * g.steps + s) * 4);
#pragma unroll
    for (int k = 0; k < kSteps; ++k) {
      f.lo[k] = f.hi[k] = i32x4{0, 0, 0, 0};
      if (s + k < s1) {
        f.lo[k] = *reinterpret_cast<const i32x4*>(x + int64_t(s + k) * XB);
        if (S::FORM == kMxE4M3) f.hi[k] = *reinterpret_cast<const i32x4*>(x + int64_t(s + k) * XB + 64);
      }
    }
  };
  f32x4 acc = {0.f, 0.f, 0.f, 0.f};
  WeightSteps now{}, next{};
  TokenSteps tokens{};
  if (s0 < s1) load_weights(now, s0);
  for (int s = s0; s < s1; s += kSteps) {
    if (!S::MIDDLE) load_tokens(tokens, s);
    if (s + kSteps < s1) load_weights(next, s + kSteps);
#pragma unroll
    for (int k = 0; k < kSteps; ++k) {
      if (s + k >= s1) break;  // (scales there are another row's, and may be NaN)
      i32x4 lo = tokens.lo[k], hi = tokens.hi[k];
      int scale = int(tokens.s[k] >> (8 * q));
      if constexpr (S::MIDDLE) quantise_step<S::FORM>(middle + (s + k) * 128, q, lane, lo, hi, scale);
      acc = mx_multiply<S::FORM, S::EXACT>(now.w[k], int(now.s[k] >> (8 * q)), lo, hi, scale, acc);
    }
    now = next;
  }
  // accumulator v of lane l: weight row 4 (l / 16) + v, token l % 16
#pragma unroll
  for (int v = 0; v < 4; ++v) sums[wave][4 * q + v][r] = acc[v];
  __syncthreads();

  const DenseEpi& e = g.epi;
  const int row = threadIdx.x / NC, c = threadIdx.x % NC, col = n0 + c;
  if (row >= g.T) return;
  float v = 0.f, u = 0.f;
#pragma unroll
  for (int k = 0; k < kWaves; ++k) {
    v += sums[k][c][row];
    if (S::DUAL) u += sums[k][NC + c][row];
  }
  if constexpr (S::DUAL) {
    g.mid[row * int64_t((g.N + 127) & ~127) + col] = col < g.N ? act_one(e.act, v) * u : 0.f;
  } else if (col < g.N) {
    if (e.bias) v += load1(e, e.bias, col);
    v = act_one(e.act, v);
    if (e.residual) v += load1(e, e.residual, row * e.ld_residual + col);
    if (e.f32) static_cast<float*>(e.out)[row * e.ld_out + col] = v;
    else static_cast<bf16_t*>(e.out)[row * e.ld_out + col] = f32_to_bf16(v);
  }
}

namespace {

template <class S> hipError_t launch(const MxArgs& g, unsigned grid, hipStream_t st) {
  hipLaunchKernelGGL(mx_stream_kernel<S>, dim3(grid), dim3(64 * kWaves), 0, st, g);
  return hipGetLastError();
}
template <int FORM, bool EXACT> hipError_t launch_form(const MxArgs& g, hipStream_t st) {
  // (dual: columns up to whole steps, the padding is written too)
  if (g.w2) return launch<MxStreamShape<FORM, true, EXACT, false>>(g, unsigned((g.N + 127) / 128 * 16), st);
  const unsigned grid = unsigned((g.N + kRows - 1) / kRows);
  return g.middle ? launch<MxStreamShape<FORM, false, EXACT, true>>(g, grid, st)
                  : launch<MxStreamShape<FORM, false, EXACT, false>>(g, grid, st);
}

}  // namespace

hipError_t launch_mx_stream(const MxArgs& g, int form, hipStream_t st) {
  if (g.T < 1 || g.T > kMxStreamTokens || g.N < 1 || g.steps < 1) return hipErrorInvalidValue;
  if (form == kMxE2M1) return launch_form<kMxE2M1, false>(g, st);
  return g.exact ? launch_form<kMxE4M3, true>(g, st) : launch_form<kMxE4M3, false>(g, st);
}

}  // namespace moe
