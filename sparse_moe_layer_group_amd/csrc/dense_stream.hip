// Dense products of few tokens (a serving step), bfloat16 and float32: the
// weights pass through once and are all that counts.
//
//   out[t][n] = epilogue(sum_k x[t][k] w[n][k])  (dual: act(x w^T) * (x w2^T))
//
// Memory-bound: a weight is used for at most 64 tokens, far below the MFMA's
// rate, so what matters is that every CU keeps enough bytes in flight.  A
// workgroup of eight waves takes 16 weight rows (dual: 8 of each matrix, the
// same columns); the waves take the contraction in turns of 128, each with the
// loads of its next turn in flight, and their sums are joined through LDS in
// wave order.  So a product of few columns still has all its contraction in
// flight at once, with no second launch.  Weights go from memory to registers
// as they lie, 16 bytes a lane at any alignment; a 16x16x32 MFMA takes 16 rows
// of them against 16 tokens.  float32 operands are split in registers into
// three bfloat16 parts (exactly) and multiplied as six MFMAs.
//
// Measured, one token, bfloat16: 2 x 2048 rows of 7168 in 13.5 us = 4.4 TB/s,
// 7168 rows of 2048 in 8.8 us = 3.3 TB/s; a launch that reads nothing takes 3.5.
// From 17 tokens on the loads of the tokens themselves, which every workgroup
// repeats, are what bounds it (32 tokens through both: 39 us, by tiles 29), in
// float32 with splitting them again in every workgroup (one token 46 us, 16 56,
// 32 79, 64 129).
#include "block.h"

namespace moe {

namespace {

constexpr int kWaves = 8;      // of a workgroup
constexpr int kTurn = 128;     // contraction of a wave's turn: four MFMA steps of 32
constexpr int kRows = 16;      // weight rows of a workgroup

// 8 consecutive elements as MFMA operands: one bfloat16 part, or three
template <typename TE> struct Part8;
template <> struct Part8<bf16_t> {
  static constexpr int N = 1;
  u32x4 raw;
  MOE_DEV void load(const bf16_t* p, int k, int K, bool inside) {
    raw = inside ? reinterpret_cast<const u32x4_at2*>(p + k)->v : load8_raw<false>(p, k, K);
  }
  template <bool> MOE_DEV void parts(bf16x8 (&o)[1]) const { o[0] = __builtin_bit_cast(bf16x8, raw); }
};
template <> struct Part8<float> {
  static constexpr int N = 3;
  float v[8];
  MOE_DEV void load(const float* p, int k, int K, bool inside) {
    if (inside) load8<true>(p, k, k + 8, v);
    else load8<false>(p, k, K, v);
  }
  template <bool ANY> MOE_DEV void parts(bf16x8 (&o)[3]) const {
    u32x4 w[3];
    split8<ANY>(v, w);
#pragma unroll
    for (int s = 0; s < 3; ++s) o[s] = __builtin_bit_cast(bf16x8, w[s]);
  }
};

template <int N> MOE_DEV f32x4 mfma_parts(const bf16x8 (&a)[N], const bf16x8 (&b)[N], f32x4 acc) {
  if (N == 3) {  // smallest terms first
    acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a[N - 1], b[0], acc, 0, 0, 0);
    acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a[0], b[N - 1], acc, 0, 0, 0);
    acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a[N / 2], b[N / 2], acc, 0, 0, 0);
    acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a[N / 2], b[0], acc, 0, 0, 0);
    acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a[0], b[N / 2], acc, 0, 0, 0);
  }
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a[0], b[0], acc, 0, 0, 0);
}

// TT: groups of 16 tokens
template <typename TE_, int TT_, bool DUAL_> struct StreamShape {
  typedef TE_ TE;
  static constexpr int TT = TT_;
  static constexpr bool DUAL = DUAL_;
};

}  // namespace

template <class S> __global__ __launch_bounds__(64 * kWaves) void dense_stream_kernel(DenseStreamArgs g) {
  typedef typename S::TE TE;
  constexpr int TT = S::TT, NC = S::DUAL ? kRows / 2 : kRows;  // output columns of a workgroup
  __shared__ float sums[kWaves][TT * 16][kRows + 1];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int n0 = blockIdx.x * NC;
  const int r = lane & 15, kq = 8 * (lane >> 4);
  // this lane's weight row and token rows; rows past the end repeat the last
  const int n = min(n0 + (S::DUAL ? r & 7 : r), g.N - 1);
  const TE* w = static_cast<const TE*>(S::DUAL && r >= 8 ? g.w2 : g.w) + int64_t(n) * g.K;
  const TE* x[TT];
#pragma unroll
  for (int i = 0; i < TT; ++i) x[i] = static_cast<const TE*>(g.x) + int64_t(min(16 * i + r, g.T - 1)) * g.ld_x;

  f32x4 acc[TT];
#pragma unroll
  for (int i = 0; i < TT; ++i) acc[i] = f32x4{0.f, 0.f, 0.f, 0.f};

  // The next turn's weights are in flight during a turn; the tokens, which the
  // caches hold, are loaded in it.  (Three turns ahead, tokens too: no faster
  // for one token, 12% slower for 16, and float32 spills from 33 on.)
  constexpr int STEPS = kTurn / 32;
  Part8<TE> wn[STEPS];
  auto fetch = [&](int k0) {
    const bool inside = k0 + kTurn <= g.K;
#pragma unroll
    for (int s = 0; s < STEPS; ++s) wn[s].load(w, k0 + 32 * s + kq, g.K, inside);
  };
  int k0 = wave * kTurn;
  if (k0 < g.K) fetch(k0);
  for (; k0 < g.K; k0 += kWaves * kTurn) {
    Part8<TE> wc[STEPS], xc[TT][STEPS];
    const bool inside = k0 + kTurn <= g.K;
#pragma unroll
    for (int s = 0; s < STEPS; ++s) {
      wc[s] = wn[s];
#pragma unroll
      for (int i = 0; i < TT; ++i) xc[i][s].load(x[i], k0 + 32 * s + kq, g.K, inside);
    }
    if (k0 + kWaves * kTurn < g.K) fetch(k0 + kWaves * kTurn);
#pragma unroll
    for (int s = 0; s < STEPS; ++s) {
      bf16x8 a[Part8<TE>::N], b[Part8<TE>::N];
      wc[s].template parts<false>(a);
#pragma unroll
      for (int i = 0; i < TT; ++i) {
        xc[i][s].template parts<false>(b);
        acc[i] = mfma_parts(a, b, acc[i]);
      }
    }
  }
  // A value that needs split8<true> and had split8<false> has left a NaN in the
  // sums, and so may others: such a wave's share once more.
  // (Asking for infinities before each turn holds all of its values at once and
  // spilled 32 registers from 33 tokens on.)
  bool again = false;
#pragma unroll
  for (int i = 0; i < TT; ++i)
#pragma unroll
    for (int v = 0; v < 4; ++v) again = again || acc[i][v] != acc[i][v];
  if (Part8<TE>::N > 1 && __builtin_amdgcn_ballot_w64(again) != 0) {
#pragma unroll
    for (int i = 0; i < TT; ++i) acc[i] = f32x4{0.f, 0.f, 0.f, 0.f};
    for (k0 = wave * kTurn; k0 < g.K; k0 += kWaves * kTurn) {
#pragma unroll 1
      for (int k = k0; k < k0 + kTurn; k += 32) {
        Part8<TE> v;
        bf16x8 a[Part8<TE>::N], b[Part8<TE>::N];
        v.load(w, k + kq, g.K, k0 + kTurn <= g.K);
        v.template parts<true>(a);
#pragma unroll
        for (int i = 0; i < TT; ++i) {
          v.load(x[i], k + kq, g.K, k0 + kTurn <= g.K);
          v.template parts<true>(b);
          acc[i] = mfma_parts(a, b, acc[i]);
        }
      }
    }
  }
  // accumulator v of lane l: weight row 4 (l / 16) + v, token l % 16
#pragma unroll
  for (int i = 0; i < TT; ++i)
#pragma unroll
    for (int v = 0; v < 4; ++v) sums[wave][16 * i + r][4 * (lane >> 4) + v] = acc[i][v];
  __syncthreads();
  for (int id = threadIdx.x; id < TT * 16 * NC; id += 64 * kWaves) {
    const int t = id / NC, c = id % NC, col = n0 + c;
    if (t >= g.T || col >= g.N) continue;
    float v = 0.f, u = 0.f;
#pragma unroll
    for (int q = 0; q < kWaves; ++q) {
      v += sums[q][t][c];
      if (S::DUAL) u += sums[q][t][kRows / 2 + c];
    }
    if (!S::DUAL && g.bias) v += to_f32(static_cast<const TE*>(g.bias)[col]);
    v = act_one(g.act, v);
    if (S::DUAL) v *= u;
    if (!S::DUAL && g.residual) v += to_f32(static_cast<const TE*>(g.residual)[t * g.ld_residual + col]);
    static_cast<TE*>(g.out)[t * g.ld_out + col] = from_f32<TE>(v);
  }
}

namespace {

template <typename TE, int TT> hipError_t launch_tokens(const DenseStreamArgs& g, hipStream_t st) {
  const unsigned nc = g.w2 ? kRows / 2 : kRows, grid = (unsigned(g.N) + nc - 1) / nc;
  if (g.w2)
    hipLaunchKernelGGL((dense_stream_kernel<StreamShape<TE, TT, true>>), dim3(grid), dim3(64 * kWaves), 0, st, g);
  else
    hipLaunchKernelGGL((dense_stream_kernel<StreamShape<TE, TT, false>>), dim3(grid), dim3(64 * kWaves), 0, st, g);
  return hipGetLastError();
}
template <typename TE> hipError_t launch_type(const DenseStreamArgs& g, hipStream_t st) {
  if (g.T <= 16) return launch_tokens<TE, 1>(g, st);
  if (g.T <= 32) return launch_tokens<TE, 2>(g, st);
  return launch_tokens<TE, 4>(g, st);
}

}  // namespace

hipError_t launch_dense_stream(const DenseStreamArgs& g, bool f32, hipStream_t st) {
  if (g.T < 1 || g.T > kStreamTokens || g.N < 1) return hipErrorInvalidValue;
  return f32 ? launch_type<float>(g, st) : launch_type<bf16_t>(g, st);
}

}  // namespace moe
