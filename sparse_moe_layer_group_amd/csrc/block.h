// Shared pieces of the operators around the expert layer (norm_kernels.hip,
// dense_gemm.hip, dense_stream.hip, block_api.cpp); not part of the C ABI.
#pragma once

#include "common.h"

namespace moe {

// ---------------------------------------------------------------- activations

// codes of enum moe_act
constexpr int kActNone = 0, kActRelu = 1, kActSilu = 2, kActGelu = 3;

// (NaN stays NaN, in the slope too, as in the others: a maximum would hide it)
MOE_DEV float relu_value(float z) { return z < 0.f ? 0.f : z; }
MOE_DEV float relu_slope(float z) { return z > 0.f ? 1.f : z <= 0.f ? 0.f : z; }
MOE_DEV float silu_slope(float z) {
  const float s = sigmoidf(z);
  return s * (1.0f + z * (1.0f - s));
}
// z Phi(z) and Phi(z) + z phi(z)
MOE_DEV float gelu_value(float z) { return 0.5f * z * erfcf(-0.70710678118654752f * z); }
MOE_DEV float gelu_slope(float z) {
  return 0.5f * erfcf(-0.70710678118654752f * z) + z * 0.39894228040143268f * expf(-0.5f * z * z);
}

// eight values become their activation, or its slope there.  One branch on the
// (uniform) kind for all eight: one for each keeps every kind's code in the way
// of every element, and the instruction fetch of an epilogue then costs more
// than its arithmetic.
template <class F> MOE_DEV void each8(float (&v)[8], F f) {
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = f(v[i]);
}
MOE_DEV void act_values(int act, float (&v)[8]) {
  if (act == kActSilu) each8(v, siluf);
  else if (act == kActGelu) each8(v, gelu_value);
  else if (act == kActRelu) each8(v, relu_value);
}
// v becomes the activation, d its slope
MOE_DEV void act_both(int act, float (&v)[8], float (&d)[8]) {
  if (act == kActSilu) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float s = sigmoidf(v[i]);
      d[i] = s * (1.0f + v[i] * (1.0f - s));
      v[i] *= s;
    }
  } else if (act == kActGelu) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float z = v[i], phi = 0.5f * erfcf(-0.70710678118654752f * z);
      d[i] = phi + z * 0.39894228040143268f * expf(-0.5f * z * z);
      v[i] = z * phi;
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      d[i] = act == kActRelu ? relu_slope(v[i]) : 1.f;
      v[i] = act == kActRelu ? relu_value(v[i]) : v[i];
    }
  }
}
MOE_DEV float act_one(int act, float z) {
  return act == kActSilu ? siluf(z) : act == kActGelu ? gelu_value(z) : act == kActRelu ? relu_value(z) : z;
}
MOE_DEV float slope_one(int act, float z) {
  return act == kActSilu ? silu_slope(z) : act == kActGelu ? gelu_slope(z) : act == kActRelu ? relu_slope(z) : 1.f;
}
MOE_DEV void act_slopes(int act, float (&v)[8]) {
  if (act == kActSilu) each8(v, silu_slope);
  else if (act == kActGelu) each8(v, gelu_slope);
  else if (act == kActRelu) each8(v, relu_slope);
  else each8(v, [](float) { return 1.f; });
}

// ---------------------------------------------------------------- 8 elements of a row

// Global memory takes vector accesses at any element's address; these types
// let the compiler use them where a row's start is aligned to its element only.
struct __attribute__((packed, aligned(2))) u32x4_at2 { u32x4 v; };
struct __attribute__((packed, aligned(4))) f32x4_at4 { f32x4 v; };

// Elements c .. c+7 of a row of n, zeros past its end.  WHOLE: n is a multiple
// of 8, so eight elements are all inside the row or all past it.
template <bool WHOLE> MOE_DEV void load8(const float* row, int c, int n, float (&v)[8]) {
  if (c + 8 <= n) {
    const f32x4 a = reinterpret_cast<const f32x4_at4*>(row + c)->v;
    const f32x4 b = reinterpret_cast<const f32x4_at4*>(row + c + 4)->v;
#pragma unroll
    for (int i = 0; i < 4; ++i) { v[i] = a[i]; v[4 + i] = b[i]; }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = !WHOLE && c + i < n ? row[c + i] : 0.f;
  }
}
MOE_DEV void unpack8(u32x4 a, float (&v)[8]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(a[i] << 16);
    v[2 * i + 1] = __uint_as_float(a[i] & 0xffff0000u);
  }
}
// the bfloat16 elements as they are, two to a register
template <bool WHOLE> MOE_DEV u32x4 load8_raw(const bf16_t* row, int c, int n) {
  if (c + 8 <= n) return reinterpret_cast<const u32x4_at2*>(row + c)->v;
  u32x4 a = {0u, 0u, 0u, 0u};
  if (!WHOLE && c < n) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t lo = c + 2 * i < n ? row[c + 2 * i] : 0u, hi = c + 2 * i + 1 < n ? row[c + 2 * i + 1] : 0u;
      a[i] = lo | (hi << 16);
    }
  }
  return a;
}
template <bool WHOLE> MOE_DEV void load8(const bf16_t* row, int c, int n, float (&v)[8]) {
  unpack8(load8_raw<WHOLE>(row, c, n), v);
}

// two float32 to a pair of bfloat16, round to nearest even (gfx950's v_cvt_pk_bf16_f32)
MOE_DEV uint32_t pack_bf16(float a, float b) {
  typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
  const bf16x2 p = {(__bf16)a, (__bf16)b};
  return __builtin_bit_cast(uint32_t, p);
}
MOE_DEV u32x4 pack8(const float (&v)[8]) {
  return u32x4{pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]), pack_bf16(v[6], v[7])};
}

template <bool WHOLE> MOE_DEV void store8(float* row, int c, int n, const float (&v)[8]) {
  if (c + 8 <= n) {
    reinterpret_cast<f32x4_at4*>(row + c)->v = f32x4{v[0], v[1], v[2], v[3]};
    reinterpret_cast<f32x4_at4*>(row + c + 4)->v = f32x4{v[4], v[5], v[6], v[7]};
  } else if (!WHOLE) {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (c + i < n) row[c + i] = v[i];
  }
}
template <bool WHOLE> MOE_DEV void store8(bf16_t* row, int c, int n, const float (&v)[8]) {
  if (c + 8 <= n) {
    reinterpret_cast<u32x4_at2*>(row + c)->v = pack8(v);
  } else if (!WHOLE) {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (c + i < n) row[c + i] = f32_to_bf16(v[i]);
  }
}

// ---------------------------------------------------------------- float32 as three bfloat16 parts

// v = part 0 + part 1 + part 2, exactly: each part is what is left, rounded to
// nearest, so part 1 is up to 2^-8 of v and part 2 up to 2^-17, of either sign,
// and the pairs of parts that a product leaves out (below 2^-24 of it) do not
// add up over a sum as truncated parts' did, which were four times as large.
// Where part 0 would round up past the largest bfloat16 it is that one.  A value
// that is not finite is part 2 alone, its others are 0: of the products that
// stand for v w, part 2 takes part in one, with w's part 0, and an infinity then
// meets neither a 0 nor a part of the other sign.  (Two infinities at the same
// place of a contraction give NaN.)
MOE_DEV bool finite(float v) { return (__float_as_uint(v) & 0x7f800000u) != 0x7f800000u; }
constexpr float kMostBf16 = 0x1.fep127f;
MOE_DEV float first_of(float v) { return __builtin_amdgcn_fmed3f(v, -kMostBf16, kMostBf16); }

// ANY: whatever the values; else the parts of one above kMostBf16 may be
// infinite and NaN
template <bool ANY> MOE_DEV void split8(const float (&v)[8], u32x4 (&o)[3]) {
  float r[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) r[i] = !ANY || finite(v[i]) ? v[i] : 0.f;
#pragma unroll
  for (int s = 0; s < 3; ++s) {
    float t[8], p[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) t[i] = !ANY || s == 1 ? r[i] : s == 0 ? first_of(r[i]) : finite(v[i]) ? r[i] : v[i];
    o[s] = pack8(t);
    unpack8(o[s], p);
#pragma unroll
    for (int i = 0; i < 8; ++i) r[i] -= p[i];
  }
}
MOE_DEV void split_any8(const float (&v)[8], u32x4 (&o)[3]) {
  float most = 0.f;  // of the magnitudes (NaN, whose parts are all NaN either way, is passed over)
#pragma unroll
  for (int i = 0; i < 8; i += 2)
    asm("v_max3_f32 %0, %1, |%2|, |%3|" : "=v"(most) : "v"(most), "v"(v[i]), "v"(v[i + 1]));
  if (__builtin_expect(__builtin_amdgcn_ballot_w64(most > kMostBf16) != 0, 0)) split8<true>(v, o);
  else split8<false>(v, o);
}
MOE_DEV void split1(float v, bf16_t (&o)[3]) {
  float r = finite(v) ? v : 0.f;
#pragma unroll
  for (int s = 0; s < 3; ++s) {
    o[s] = f32_to_bf16(s == 0 ? first_of(r) : s == 2 && !finite(v) ? v : r);
    r -= bf16_to_f32(o[s]);
  }
}

// v plus another lane's v (a move within 16-lane rows; every source is inside)
template <int CTRL> MOE_DEV float add_dpp(float v) {
  return v + __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(v), CTRL, 0xf, 0xf, true));
}
// ---------------------------------------------------------------- norm (norm_kernels.hip)

// One call's arguments; row strides in elements.  Absent tensors are NULL.
struct NormArgs {
  const void *residual, *branch, *du, *dh;
  const void *w_post, *b_post, *w_pre, *b_pre, *gate;
  void *u, *h;                       // forward outputs
  void *d_residual, *d_branch;       // backward outputs
  void *dw_post, *db_post, *dw_pre, *db_pre, *dgate;
  float* part;                       // [4][workgroups][H]: sums of dw_post, db_post, dw_pre, db_pre
  float* gpart;                      // [2 workers][H]: of the gate rows that workers share
  int64_t ld_residual, ld_branch, ld_u, ld_h, ld_du, ld_dh, ld_dr, ld_db;
  int64_t T;
  int H, gate_rows, layer;           // gate_rows 0: no gate
  int workers, options, partials;    // set by the launchers
  float eps, scale;
};
int norm_backward_workers(int64_t T, int H);
hipError_t launch_norm_forward(const NormArgs& a, bool bf16, hipStream_t st);
hipError_t launch_norm_backward(const NormArgs& a, bool bf16, hipStream_t st);
constexpr int kNormMaxHidden = 16384;

// ---------------------------------------------------------------- dense products (dense_gemm.hip)

// What becomes of a product's float32 sums v (and u, the second product of a
// dual call), 8 columns of a row at a time.
enum DenseEpiMode {
  kEpiOut = 0,    // out = residual + act(v + bias)
  kEpiGated,      // p0 = act(v) u
  kEpiKeep,       // g = v, u = u (float32)
  kEpiGatedBack,  // v = dM: p0 = dM u act'(g), p1 = dM act(g), p2 = act(g) u
  kEpiActBack     // p0 = dy act'(v + bias)
};
struct DenseEpi {
  int mode, act, f32;       // f32: bias, residual, out and dy are float32 (else bfloat16)
  int64_t M;
  int N;                    // output columns
  const void *bias, *residual, *dy;
  void* out;
  int64_t ld_residual, ld_out, ld_dy;
  bf16_t *p0, *p1, *p2;     // staged operands: [f32 ? 3 : 1][M][ld_p], columns N .. ld_p up to 8 written as 0
  int64_t plane, ld_p;      // elements between planes, and rows
  float *g, *u;             // [M][ld_p]
  float* sums;              // kEpiActBack: [row tiles x 2][N], sums over the rows, or NULL (not wanted).  A split
                            // contraction leaves the results themselves in its first part instead.
};

// out[m][n] = sum over segments and k of A[m][k] B[n][k], each operand given
// per segment.  Layout: a k-contiguous operand is [rows][ld], a k-slow one
// [k][ld].  Operands are bfloat16, 16-byte aligned, ld % 8 == 0, and a
// k-contiguous one holds zeros from K up to the next multiple of 8.
constexpr int kMaxSegments = 12;
enum DenseLayout { kNT = 0, kNN = 1, kTN = 2 };  // A, B: k-contiguous (N... T) as in A B^T, A B, A^T B
struct DenseArgs {
  const bf16_t* a[kMaxSegments];
  const bf16_t* b[kMaxSegments];
  const bf16_t* b2[kMaxSegments];  // dual (kNT only): the second product's B
  int64_t lda, ldb;
  int64_t M, K;                    // K of one segment
  int N, segments, dual;
  int split, steps_per_split;      // set by the launcher
  float* part;                     // (set by the launcher) split > 1: [split][1 + dual][M][ld_part]
  int64_t ld_part;
  DenseEpi epi;
};
// Up to three products of one layout, mode, contraction and M N go in one
// launch (the gate, up and down matrices' gradients).
constexpr int kMaxGroup = 4;  // these and a data gradient
struct DenseGroup { DenseArgs g[kMaxGroup]; };
// Room for the sums of a split contraction: of this product (thin: it may take the
// 64 x 32 tile); and enough for it with any smaller M, or any smaller K (A^T B)
size_t dense_part_bytes(int64_t M, int N, int64_t K, int segments, int dual, int count, bool thin);
size_t dense_part_most(int64_t M, int N, int64_t K, int segments, int dual, int count);
size_t dense_part_most_deep(int64_t M, int N, int64_t K, int segments, int count);
hipError_t launch_dense(const DenseGroup& group, int count, int layout, float* part, hipStream_t st);
hipError_t launch_dense_gradients(const DenseArgs& data, const DenseGroup& weights, int count, float* part,
                                  hipStream_t st);

// ---------------------------------------------------------------- few tokens (dense_stream.hip)

// out[t][n] = residual + act(x w^T + bias), or with w2: act(x w^T) * (x w2^T),
// all of one type; w and w2 are packed [N][K]
struct DenseStreamArgs {
  const void *x, *w, *w2, *bias, *residual;
  void* out;
  int64_t ld_x, ld_residual, ld_out;
  int T, N, K, act;
};
constexpr int kStreamTokens = 64;
hipError_t launch_dense_stream(const DenseStreamArgs& a, bool f32, hipStream_t st);

// ---------------------------------------------------------------- operands

// Planes of operands, all in one launch: dst [f32 ? 3 : 1][rows][ld_dst] with
// zeros past cols.  float32 values are split exactly into three bfloat16 parts.
struct PackJob {
  const void* src;
  int64_t ld_src, rows;
  int cols;
  bf16_t* dst;
  int64_t ld_dst;
};
constexpr int kMaxPacks = 5;
struct PackJobs { PackJob j[kMaxPacks]; };
hipError_t launch_dense_pack(const PackJobs& jobs, int count, bool f32, hipStream_t st);

// Sums over rows: out[n] = sum over r of src[r][n], src bfloat16 or float32 (src_f32);
// and a product with kEpiActBack with those of its results, unrounded, as dbias
// (NULL: not wanted).  sums: dense_sums_bytes of room.
size_t dense_sums_bytes(int64_t rows, int cols);
hipError_t launch_dense_colsum(const void* src, bool src_f32, int64_t ld, int64_t rows, int cols, void* out, bool f32,
                               float* sums, hipStream_t st);
hipError_t launch_dense_act_back(const DenseArgs& g, void* dbias, float* sums, float* part, hipStream_t st);

}  // namespace moe
