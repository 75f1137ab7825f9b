// What the tiled products (dense_gemm.hip, mx_gemm.hip) share.
#pragma once

#include "block.h"
#include "lds_async.h"

namespace moe {

typedef __attribute__((address_space(3))) uint8_t lds_u8;
typedef __attribute__((address_space(3))) f32x4 lds_f32x4;

// s_waitcnt immediates: vmcnt(0) and lgkmcnt(0); vmcnt(n)
constexpr int kWaitAll = 0x0070;
constexpr int wait_copies(int n) { return (n & 15) | ((n >> 4) << 14) | 0x70 | 0xf00; }

// Between other accesses to accumulators and products, either way round: no
// instruction on an accumulator passes it.
template <int M, int N> MOE_DEV void settle(f32x4 (&acc)[M][N]) {
#pragma unroll
  for (int k = 0; k < 2; ++k) {
#pragma unroll
    for (int i = 0; i < M; ++i)
#pragma unroll
      for (int j = 0; j < N; ++j) asm volatile("" : "+a"(acc[i][j]));
    if (k == 0) asm volatile("s_nop 15\n\ts_nop 7");
  }
}

// ---------------------------------------------------------------- epilogue

// v as staged planes at p + offset (one, rounded to bfloat16; or three whose sum is v)
MOE_DEV void store_planes(const DenseEpi& e, bf16_t* p, int64_t offset, const float (&v)[8]) {
  bf16_t* at = p + offset;
  if (!e.f32) {
    *reinterpret_cast<u32x4*>(at) = pack8(v);
    return;
  }
  u32x4 o[3];
  split_any8(v, o);
#pragma unroll
  for (int s = 0; s < 3; ++s) *reinterpret_cast<u32x4*>(at + s * e.plane) = o[s];
}

MOE_DEV void store_f32(float* p, const float (&v)[8]) {
  reinterpret_cast<f32x4*>(p)[0] = f32x4{v[0], v[1], v[2], v[3]};
  reinterpret_cast<f32x4*>(p)[1] = f32x4{v[4], v[5], v[6], v[7]};
}

// columns n .. n+7 of rows m, m + step, ... of a matrix of the call's type.
// INSIDE: all of them are inside the matrix (else zeros stand for columns past N).
template <bool INSIDE, int R>
MOE_DEV void load_rows(const DenseEpi& e, const void* p, int64_t ld, int64_t m, int step, int n, float (&v)[R][8]) {
  const int end = INSIDE ? n + 8 : e.N;
  const int64_t first = m * ld, next = step * ld;  // one wide product for all rows
  if (e.f32) {
#pragma unroll
    for (int k = 0; k < R; ++k) load8<INSIDE>(static_cast<const float*>(p) + (first + k * next), n, end, v[k]);
  } else {
    u32x4 raw[R];
#pragma unroll
    for (int k = 0; k < R; ++k)
      raw[k] = load8_raw<INSIDE>(static_cast<const bf16_t*>(p) + (first + k * next), n, end);
#pragma unroll
    for (int k = 0; k < R; ++k) unpack8(raw[k], v[k]);
  }
}

// the bias of columns n .. n+7, or zeros
template <int MODE, bool INSIDE> MOE_DEV void load_bias(const DenseEpi& e, int n, float (&b)[1][8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) b[0][i] = 0.f;
  if ((MODE == kEpiOut || MODE == kEpiActBack) && e.bias) load_rows<INSIDE, 1>(e, e.bias, 0, 0, 0, n, b);
}

// Columns n .. n+7 (n % 8 == 0, n < N) of the R rows m, m + step, ...: their
// loads are issued together, then the arithmetic, then their stores.  RESIDUAL:
// e.residual is there.  (Asked at both its load and its use, it leaves the
// compiler a path with loads that nothing waited for, and it then waits for all
// memory operations, the stores too, before the next rows.)  early: the rows of
// the residual or upstream gradient, where they were loaded before.  total:
// kEpiActBack's results are added to it, as they are before they are rounded,
// and left in v.  STREAM: kEpiOut's rows go past the caches.
template <int MODE, bool INSIDE, bool RESIDUAL, int R, bool STREAM = false>
MOE_DEV void dense_rows(const DenseEpi& e, int64_t m, int step, int n, float (&v)[R][8], float (&u)[R][8],
                        const float (&b)[1][8], float (&total)[8], const u32x4* early = nullptr) {
  float x[R][8];  // residual, upstream gradient or gate projection
  if (early != nullptr) {
#pragma unroll
    for (int k = 0; k < R; ++k) unpack8(early[k], x[k]);
  } else if (RESIDUAL) {
    load_rows<INSIDE, R>(e, e.residual, e.ld_residual, m, step, n, x);
  } else if (MODE == kEpiActBack) {
    load_rows<INSIDE, R>(e, e.dy, e.ld_dy, m, step, n, x);
  }
  if (MODE == kEpiGatedBack) {
#pragma unroll
    for (int k = 0; k < R; ++k) {
      const int64_t o = m * e.ld_p + n + k * (step * e.ld_p);
      load8<true>(e.g + o, 0, 8, x[k]);
      load8<true>(e.u + o, 0, 8, u[k]);
    }
  }
  if (!INSIDE) {  // sums of columns past N are of whatever lies there
#pragma unroll
    for (int k = 0; k < R; ++k)
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        v[k][i] = n + i < e.N ? v[k][i] : 0.f;
        u[k][i] = n + i < e.N ? u[k][i] : 0.f;
      }
  }
  if (MODE == kEpiOut || MODE == kEpiActBack) {
#pragma unroll
    for (int k = 0; k < R; ++k)
#pragma unroll
      for (int i = 0; i < 8; ++i) v[k][i] += b[0][i];
  }
  if (MODE == kEpiOut) {
    if (e.act != kActNone) {
#pragma unroll
      for (int k = 0; k < R; ++k) act_values(e.act, v[k]);
    }
    if (RESIDUAL) {
#pragma unroll
      for (int k = 0; k < R; ++k)
#pragma unroll
        for (int i = 0; i < 8; ++i) v[k][i] += x[k][i];
    }
    const int end = INSIDE ? n + 8 : e.N;
    const int64_t first = m * e.ld_out, next = step * e.ld_out;
    if (e.f32) {
#pragma unroll
      for (int k = 0; k < R; ++k) store8<INSIDE, STREAM>(static_cast<float*>(e.out) + (first + k * next), n, end, v[k]);
    } else {
#pragma unroll
      for (int k = 0; k < R; ++k) store8<INSIDE, STREAM>(static_cast<bf16_t*>(e.out) + (first + k * next), n, end, v[k]);
    }
    return;
  }
#pragma unroll
  for (int k = 0; k < R; ++k) {
    const int64_t o = m * e.ld_p + n + k * (step * e.ld_p);
    if (MODE == kEpiActBack) {
      act_slopes(e.act, v[k]);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        v[k][i] *= x[k][i];
        total[i] += v[k][i];
      }
      store_planes(e, e.p0, o, v[k]);
    } else if (MODE == kEpiGated) {
      act_values(e.act, v[k]);
#pragma unroll
      for (int i = 0; i < 8; ++i) v[k][i] *= u[k][i];
      store_planes(e, e.p0, o, v[k]);
    } else if (MODE == kEpiKeep) {
      store_f32(e.g + o, v[k]);
      store_f32(e.u + o, u[k]);
    } else {
      float s[8], d[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) s[i] = x[k][i];
      act_both(e.act, s, x[k]);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        d[i] = v[k][i] * s[i];
        s[i] *= u[k][i];
        x[k][i] *= v[k][i] * u[k][i];
      }
      store_planes(e, e.p0, o, x[k]);
      store_planes(e, e.p1, o, d);
      store_planes(e, e.p2, o, s);
    }
  }
}

template <int MODE, bool INSIDE, int R, bool STREAM = false>
MOE_DEV void dense_epilogue(const DenseEpi& e, int64_t m, int step, int n, float (&v)[R][8], float (&u)[R][8],
                            const float (&b)[1][8], float (&total)[8]) {
  if (MODE == kEpiOut && e.residual) dense_rows<MODE, INSIDE, true, R, STREAM>(e, m, step, n, v, u, b, total);
  else dense_rows<MODE, INSIDE, false, R, STREAM>(e, m, step, n, v, u, b, total);
}

// one element of a matrix of the call's type
MOE_DEV float load1(const DenseEpi& e, const void* p, int64_t at) {
  return e.f32 ? static_cast<const float*>(p)[at] : bf16_to_f32(static_cast<const bf16_t*>(p)[at]);
}

// ---------------------------------------------------------------- tiles

// Workgroup b's tile: the ids are dealt to the XCDs in turn, so each XCD takes
// a contiguous share of the tiles, in bands of 8 row tiles whose column tiles
// follow each other: the workgroups of one XCD then share their operands in
// its L2.
MOE_DEV void tile_of(int b, int n_tiles, int mt, int nt, int& im, int& in) {
  const int per = n_tiles >> 3, more = n_tiles & 7, x = b & 7;
  const int id = x * per + min(x, more) + (b >> 3);
  const int band = id / (8 * nt), first = band * 8, rows = min(8, mt - first);
  const int at = id - first * nt;
  in = rows == 8 ? at >> 3 : at / rows;
  im = first + at - in * rows;
}

}  // namespace moe
