// Dense matrix products of the projections and of the gated feed-forward
// block, forward and backward, in bfloat16 with float32 sums.
//
// One kernel serves the three layouts a layer needs: A B^T (forward: tokens
// times weight rows), A B (data gradients: weights read along their slow
// dimension) and A^T B (weight gradients: both operands along their slow
// dimension, the tokens).  A dual product takes two B matrices at once (the
// gate and up projections), so their elementwise product is formed from the
// two accumulators.  float32 operands come as three bfloat16 planes, hi + mid
// + lo exactly, and a product as six segments of the contraction (all pairs but
// those below 2^-24 of the product, which is float32's own rounding).
//
// Bound by the matrix cores, and at that by power: a loop of nothing but MFMAs
// sustains 2.0 PFLOP/s with 16x16x32 blocks and 1.8 with 32x32x16 on values of
// normal distribution, and what copies and LDS reads draw comes off the clock.
// So the tile is the largest that the registers hold (four waves in 2 x 2, each
// 128 x 128 with its 256 accumulator registers, one workgroup a CU): it reads
// the fewest bytes from LDS and L2 per MFMA.  Smaller tiles take over where
// there are too few large ones (dense_plan).
//
// The loop.  Workgroup tile TM x TN, contraction in steps of 64 through rings of
// LDS stages filled by buffer_load ... lds copies, issued two to five steps
// ahead; fragments are read one slice of 32 ahead; copies, reads and the next
// step's addresses lie between the MFMAs, one to a gap, as a gap hides three
// instructions (the same work bunched at a step's end cost 260 of 2048 cycles);
// one barrier a step.  A k-contiguous operand is staged as rows of 64 (chunk c
// of row r at c ^ (r & 7)), a k-slow one as k-rows of TM or TN columns, read
// with the transposing ds_read_b64_tr_b16; neither has bank conflicts.
//
// Measured, bfloat16, M x N x K, operands changing from call to call (the
// library's product, which has no epilogue, in brackets): 8192 x 4096 x 7168 318
// us = 1.51 PFLOP/s (306), 4096 x 7168 x 7168 296 us (288), 8192 x 7168 x 2048
// 191 us (170 to 176), 4096 x 2048 x 7168 113 us (102).  Counters for the first:
// MFMAs busy 76% of the cycles at 1.80 GHz; 82% without copies and reads.  What
// is left is 4 us before a tile's first MFMA and 8 us for its epilogue, with
// nothing to overlap them: a workgroup that went on to its next tile instead was
// slower (its loop had waits that depend on the tile), so was an epilogue without
// LDS (rows of 64 bytes a store: 8192 x 7168 x 2048 198 -> 205 us).
//
// Bounds.  An operand's buffer resource starts at the step's own first element
// and ends with the matrix, so rows past the end read as zero without a
// comparison and offsets stay small however large the matrix is; what lies
// past the end of the contraction inside a k-contiguous row is masked by an
// offset beyond every resource.
#include <type_traits>

#include "dense_tiles.h"

namespace moe {

namespace {

constexpr int BK = 64;
constexpr uint32_t kBeyond = 0x80000000u;  // past every resource (they end below 2^31)

typedef short v4i16 __attribute__((ext_vector_type(4)));
typedef short v8i16 __attribute__((ext_vector_type(8)));
typedef __attribute__((address_space(3))) v4i16 lds_v4i16;

// position of 16-byte chunk c in k-row r of RL columns: the eight k-rows that
// two lane groups of a transposed read take together hit distinct banks
template <int RL> MOE_DEV int kswz(int r, int c) {
  return c ^ (RL >= 128 ? ((r & 3) << 1) ^ (r & 8) : ((r & 2) << 1) ^ ((r & 8) >> 2));
}

// 8 k of row `row` (k-contiguous stage of rows of 64)
MOE_DEV bf16x8 row_frag(const bf16_t* st, int row, int chunk) {
  return *reinterpret_cast<const bf16x8*>(st + row * BK + ((chunk ^ (row & 7)) << 3));
}

// columns i0 .. i0+15, k kbase .. kbase+31 of a k-row stage of RL columns:
// lane l gets column i0 + l%16, k = kbase + 8 (l/16) .. +7
template <int RL> MOE_DEV bf16x8 tr_frag(const bf16_t* st, int kbase, int i0, int lane) {
  const int g = lane >> 4, s = lane & 15;
  const int col = i0 + 4 * (s & 3);
  v4i16 h[2];
#pragma unroll
  for (int q = 0; q < 2; ++q) {
    const int k = kbase + 8 * g + 4 * q + (s >> 2);
    const bf16_t* p = st + k * RL + (kswz<RL>(k, col >> 3) << 3) + (col & 7);
    h[q] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4i16*)((__attribute__((address_space(3))) bf16_t*)p));
  }
  return __builtin_bit_cast(bf16x8, __builtin_shufflevector(h[0], h[1], 0, 1, 2, 3, 4, 5, 6, 7));
}

// acc += a b.  Written as assembly to update the accumulator where it lies: the
// builtin's result may go to other registers, and with all 256 of them taken by
// accumulators this compiler moves 190 of them about and spills 12 a step.  It
// does not know of a wait that such a product needs, so one is made before the
// first and after the last (settle).  Operands come straight from LDS reads,
// whose waits it does know of.
MOE_DEV void multiply_add(f32x4& acc, bf16x8 a, bf16x8 b) {
  asm volatile("v_mfma_f32_16x16x32_bf16 %0, %1, %2, %0" : "+a"(acc) : "v"(a), "v"(b));
}
// ---------------------------------------------------------------- one element's epilogue

// One element's planes
MOE_DEV void store_plane1(const DenseEpi& e, bf16_t* p, int64_t offset, float v) {
  if (!e.f32) {
    p[offset] = f32_to_bf16(v);
    return;
  }
  bf16_t o[3];
  split1(v, o);
#pragma unroll
  for (int s = 0; s < 3; ++s) p[offset + s * e.plane] = o[s];
}

// The epilogue of one element, for a join whose lanes have one each.  Columns
// from N to the next multiple of 8 are staged as zeros.  kEpiActBack leaves its
// unrounded result in v.
template <int MODE> MOE_DEV void dense_epilogue1(const DenseEpi& e, int64_t m, int n, float& v, float u) {
  const bool in = n < e.N;
  if (MODE == kEpiOut) {
    if (!in) return;
    v = act_one(e.act, e.bias ? v + load1(e, e.bias, n) : v);
    if (e.residual) v += load1(e, e.residual, m * e.ld_residual + n);
    if (e.f32) static_cast<float*>(e.out)[m * e.ld_out + n] = v;
    else static_cast<bf16_t*>(e.out)[m * e.ld_out + n] = f32_to_bf16(v);
    return;
  }
  const int64_t o = m * e.ld_p + n;
  if (MODE == kEpiKeep) {
    e.g[o] = v;
    e.u[o] = u;
  } else if (MODE == kEpiGated) {
    store_plane1(e, e.p0, o, in ? act_one(e.act, v) * u : 0.f);
  } else if (MODE == kEpiActBack) {
    if (in) {
      if (e.bias) v += load1(e, e.bias, n);
      v = slope_one(e.act, v) * load1(e, e.dy, m * e.ld_dy + n);
    } else {
      v = 0.f;
    }
    store_plane1(e, e.p0, o, v);
  } else {
    const float g = e.g[o], w = e.u[o], s = act_one(e.act, g);
    store_plane1(e, e.p0, o, in ? v * w * slope_one(e.act, g) : 0.f);
    store_plane1(e, e.p1, o, in ? v * s : 0.f);
    store_plane1(e, e.p2, o, in ? s * w : 0.f);
  }
}

// ---------------------------------------------------------------- the product

// AHEAD: steps from a copy to its use.  A takes AHEAD + 1 LDS stages and B AHEAD;
// as many as fit with one workgroup of the largest tile on a CU, two of others.
template <int LAYOUT_, int MODE_, int TM_, int TN_> struct DenseShape {
  static constexpr int LAYOUT = LAYOUT_, MODE = MODE_, TM = TM_, TN = TN_;
  static constexpr bool DUAL = MODE == kEpiGated || MODE == kEpiKeep;
  static constexpr int AHEAD = ((TM == 256 ? 160 : TN == 32 ? 70 : 80) * 1024 - TM * BK * 2) / ((TM + TN) * BK * 2);
  static constexpr int LDS = ((AHEAD + 1) * TM + AHEAD * TN) * BK * 2;
  static_assert(AHEAD >= 2, "B's stage is refilled a step before its use");
};

constexpr int kThreads = 256;  // four waves, 2 x 2

// This workgroup's product (blockIdx.z), read where the kernel's arguments lie:
// indexing the by-value copy makes this compiler keep one on the stack.
MOE_DEV const DenseArgs& group_args() {
  typedef const __attribute__((address_space(4))) DenseGroup* Args;
  return ((const DenseGroup*)(Args)__builtin_amdgcn_kernarg_segment_ptr())->g[blockIdx.z];
}

// v[0] becomes the sum over a lane octet of column `share`
MOE_DEV void scatter_sum(float (&v)[8], int share) {
#pragma unroll
  for (int half = 4; half >= 1; half >>= 1) {
    const bool upper = (share & half) != 0;
#pragma unroll
    for (int i = 0; i < half; ++i) {
      const float keep = upper ? v[i + half] : v[i], give = upper ? v[i] : v[i + half];
      v[i] = keep + __shfl_xor(give, half, 8);
    }
  }
}

// For kernels of more than one shape
template <class S> MOE_DEV void dense_tile() {
#include "dense_tile.inc"
}

}  // namespace

template <class S> __global__ __launch_bounds__(kThreads, 1) void dense_gemm_kernel(DenseGroup) {
#include "dense_tile.inc"
}

// Product 0 as shape S, the others, whose contraction is whole, as shape P
template <class S, class P> __global__ __launch_bounds__(kThreads, 1) void dense_pair_kernel(DenseGroup) {
  if (blockIdx.z == 0) dense_tile<S>();
  else if (blockIdx.y == 0) dense_tile<P>();
}

// Sums of a split contraction and the epilogue on them, eight columns of a row
// by one lane (SHARES 1) or, where that would leave most of the chip idle, by
// eight (SHARES 8): lane k then adds up the parts k, k + 8, ... of all eight
// columns, so that every part is in flight at once, the lanes' sums are added
// in a fixed tree that leaves column k with lane k, and each lane finishes its
// one element.  Where kEpiActBack's sums over the rows are wanted, its results
// take the place of the first part's, which only these lanes have read.
template <int MODE, int SHARES> __global__ __launch_bounds__(256) void dense_join_kernel(DenseGroup group) {
  constexpr bool DUAL = MODE == kEpiGated || MODE == kEpiKeep;
  const DenseArgs& g = group_args();
  const int nc = (g.N + 7) / 8;
  // (a product of at most 1024 tiles: its pieces fit 32 bits)
  const uint32_t id = (blockIdx.x * 256 + threadIdx.x) / SHARES, row = id / uint32_t(nc);
  const int share = threadIdx.x % SHARES;
  const int64_t m = row;
  if (m >= g.M) return;  // all of a piece's lanes
  const int n = int(id - row * nc) * 8;
  float v[1][8], u[1][8];
#pragma unroll
  for (int i = 0; i < 8; ++i) v[0][i] = u[0][i] = 0.f;
  const int64_t step = g.M * g.ld_part;
#pragma unroll 4
  for (int s = share; s < g.split; s += SHARES) {
    const float* p = g.part + s * (DUAL ? 2 : 1) * step + m * g.ld_part + n;
    float x[8], y[8];
    load8<true>(p, 0, 8, x);
    if (DUAL) load8<true>(p + step, 0, 8, y);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      v[0][i] += x[i];
      if (DUAL) u[0][i] += y[i];
    }
  }
  if (SHARES == 1) {
    float b[1][8], total[8] = {};
    load_bias<MODE, false>(g.epi, n, b);
    dense_epilogue<MODE, false, 1>(g.epi, m, 0, n, v, u, b, total);
    if (MODE == kEpiActBack && g.epi.sums) store_f32(g.part + m * g.ld_part + n, v[0]);
  } else {
    // halves are exchanged: lanes whose bit is set keep the upper columns
    scatter_sum(v[0], share);
    if (DUAL) scatter_sum(u[0], share);
    dense_epilogue1<MODE>(g.epi, m, n + share, v[0][0], u[0][0]);
    if (MODE == kEpiActBack && g.epi.sums) g.part[m * g.ld_part + n + share] = v[0][0];
  }
}

// ---------------------------------------------------------------- operands

// Eight columns a thread, blockIdx.y the job.  cols .. ld_dst are written as zeros.
template <typename TE> __global__ __launch_bounds__(256) void dense_pack_kernel(PackJobs jobs) {
  typedef const __attribute__((address_space(4))) PackJobs* Args;
  const PackJob& j = ((const PackJobs*)(Args)__builtin_amdgcn_kernarg_segment_ptr())->j[blockIdx.y];
  const int64_t per = j.ld_dst / 8, all = j.rows * per;
  for (int64_t id = int64_t(blockIdx.x) * 256 + threadIdx.x; id < all; id += int64_t(gridDim.x) * 256) {
    const int64_t r = id / per;
    const int c = int(id - r * per) * 8;
    float v[8];
    load8<false>(static_cast<const TE*>(j.src) + r * j.ld_src, c, j.cols, v);
    DenseEpi e{};
    e.f32 = sizeof(TE) == 4;
    e.plane = j.rows * j.ld_dst;
    store_planes(e, j.dst, r * j.ld_dst + c, v);
  }
}

// Column sums.  A workgroup takes 256 columns, 8 a thread, and a range of rows
// in 8 shares (share k: every eighth row from the k-th), joined in share order.
constexpr int kSumRows = 64;  // rows of a workgroup
template <typename TE>
__global__ __launch_bounds__(256) void dense_colsum_kernel(const TE* src, int64_t ld, int64_t rows, int cols,
                                                           float* part) {
  __shared__ float acc[8][256];
  const int lane = threadIdx.x & 31, share = threadIdx.x >> 5;
  const int c = blockIdx.y * 256 + lane * 8;
  const int64_t r0 = int64_t(blockIdx.x) * kSumRows;
  const int64_t r1 = r0 + kSumRows < rows ? r0 + kSumRows : rows;
  float s[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) s[i] = 0.f;
#pragma unroll 8
  for (int64_t r = r0 + share; r < r1; r += 8) {
    float v[8];
    load8<false>(src + r * ld, c, cols, v);
#pragma unroll
    for (int i = 0; i < 8; ++i) s[i] += v[i];
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) acc[share][lane * 8 + i] = s[i];
  __syncthreads();
  float t = 0.f;
#pragma unroll
  for (int k = 0; k < 8; ++k) t += acc[k][threadIdx.x];
  const int col = blockIdx.y * 256 + threadIdx.x;
  if (col < cols) part[int64_t(blockIdx.x) * cols + col] = t;
}
// A workgroup takes 32 columns and 32 shares of the partial rows, joined in share order.
template <typename TE>
__global__ __launch_bounds__(1024) void dense_colsum_join_kernel(const float* part, int64_t n, int cols, TE* out) {
  __shared__ float acc[32][33];
  const int lane = threadIdx.x & 31, share = threadIdx.x >> 5;
  const int col = blockIdx.x * 32 + lane;
  float t = 0.f;
  if (col < cols) {
#pragma unroll 4
    for (int64_t i = share; i < n; i += 32) t += part[i * cols + col];
  }
  acc[share][lane] = t;
  __syncthreads();
  if (share == 0 && col < cols) {
    t = 0.f;
#pragma unroll
    for (int k = 0; k < 32; ++k) t += acc[k][lane];
    out[col] = from_f32<TE>(t);
  }
}

// ---------------------------------------------------------------- launches

namespace {

struct DensePlan {
  int tile;         // TN, and TM from 64 on (dual: at least 128 columns)
  int split, steps;
};

int64_t tiles_of(int64_t M, int64_t N, int dual, int tile) {
  const int64_t nc = dual ? std::max(tile, 128) / 2 : tile, rows = std::max(tile, 64);
  return ((M + rows - 1) / rows) * ((N + nc - 1) / nc);
}

// What a step of the contraction takes on a CU, and what a tile takes besides
// (its first copies and its epilogue), in microseconds, with one workgroup and
// with two on the CU.  Measured on A B^T products of 16 to 8192 rows, 200 to
// 7168 columns and contractions of 512 to 16384, every tile and split of each:
// the sum below is within 10% of most of them and the choice it makes within
// 10% of the best.  A B, A^T B and the epilogues that read and write more take
// the same figures, which are too low for some (the gated backward of 4096 x 2048
// x 7168 by 128 x 128: 110 us here, 134 measured).
struct TileCost {
  int tile, per_cu;
  double step[2], once;
};
constexpr TileCost kTileCosts[] = {{256, 1, {1.25, 1.25}, 14.0}, {128, 2, {0.53, 0.95}, 4.0},
                                   {64, 2, {0.30, 0.41}, 2.5}, {32, 2, {0.25, 0.35}, 2.5}};
constexpr double kJoinOnce = 5.5, kJoinBytesPerUs = 4.5e6;  // of a split contraction's second launch

// Tile and contraction split of a product: what costs least.  The large tile
// moves half the operand bytes of the next for the same product and reaches
// the highest rate, the small ones and the split fill the chip where there are
// few tiles, and every split is paid for with its sums' way through memory.
// narrow: the 64 x 32 tile is there, for forward products of few tokens, whose
// weights should pass through as many CUs as there are (50 tokens by 7168 rows
// of 2048: 10.8 us against 13.1 by what the other tiles and splits give).
// M counts in whole 64 rows, so that one plan holds for each 64 (dense_part_most).
constexpr int kSplits[] = {1, 2, 3, 4, 6, 8, 12, 16};
constexpr int kSplitGroups = 1024;  // a split leaves at most so many workgroups
bool narrow(int layout, int mode) { return layout == kNT && mode == kEpiOut; }
DensePlan dense_plan(int64_t M, int N, int64_t K, int segments, int dual, int count, bool narrow) {
  const int64_t steps = (K + BK - 1) / BK * segments, rows = (M + 63) & ~int64_t(63);
  DensePlan best{};
  double least = 0;
  for (const TileCost& c : kTileCosts) {
    if (c.tile == 32 && !narrow) break;
    const int64_t tiles = tiles_of(M, N, dual, c.tile) * count;
    for (int split : kSplits) {
      if (split > 1 && (steps < 4 * split || tiles * split > kSplitGroups)) break;
      const int64_t per = (steps + split - 1) / split, used = (steps + per - 1) / per;
      const int64_t groups = tiles * used, slots = int64_t(256) * c.per_cu;
      const int64_t rest = groups % slots;  // after the full turns of the chip
      double t = double(groups / slots) * (double(per) * c.step[c.per_cu - 1] + c.once);
      if (rest > 0) t += double(per) * c.step[rest > 256 ? 1 : 0] + c.once;
      if (used > 1)
        t += kJoinOnce + 8.0 * double(used) * double(count) * double(rows) * N * (dual ? 2 : 1) / kJoinBytesPerUs;
      if (best.tile == 0 || t < least) {
        least = t;
        best = DensePlan{c.tile, int(used), int(per)};
      }
    }
  }
  return best;
}

template <class S> int64_t tiles_of(const DenseArgs& g) {
  constexpr int NCOL = S::DUAL ? S::TN / 2 : S::TN;
  return ((g.M + S::TM - 1) / S::TM) * ((g.N + NCOL - 1) / NCOL);
}

hipError_t launch_kernel(void (*kernel)(DenseGroup), int lds, int64_t tiles, const DenseGroup& group, int count,
                         hipStream_t st) {
  if (tiles * kThreads >= (int64_t(1) << 32)) return hipErrorInvalidValue;  // of a grid dimension
  const hipError_t err =
      hipFuncSetAttribute(reinterpret_cast<const void*>(kernel), hipFuncAttributeMaxDynamicSharedMemorySize, lds);
  if (err != hipSuccess) return err;
  hipLaunchKernelGGL(kernel, dim3(unsigned(tiles), unsigned(group.g[0].split), unsigned(count)), dim3(kThreads), lds,
                     st, group);
  return hipGetLastError();
}

template <class S> hipError_t launch_shape(const DenseGroup& group, int count, hipStream_t st) {
  int64_t tiles = 0;
  for (int i = 0; i < count; ++i) tiles = std::max(tiles, tiles_of<S>(group.g[i]));
  return launch_kernel(&dense_gemm_kernel<S>, S::LDS, tiles, group, count, st);
}

template <int LAYOUT, int MODE> hipError_t launch_narrow(const DenseGroup& group, int count, hipStream_t st) {
  if constexpr (LAYOUT == kNT && MODE == kEpiOut)
    return launch_shape<DenseShape<LAYOUT, MODE, 64, 32>>(group, count, st);
  else
    return hipErrorInvalidValue;
}

template <int MODE> hipError_t launch_join(const DenseGroup& group, int count, hipStream_t st) {
  int64_t pieces = 0;
  for (int i = 0; i < count; ++i) pieces = std::max(pieces, group.g[i].M * ((group.g[i].N + 7) / 8));
  // eight lanes a piece where one would not fill the chip
  if (pieces * count < 65536)
    hipLaunchKernelGGL((dense_join_kernel<MODE, 8>), dim3(unsigned((pieces + 31) / 32), 1, unsigned(count)), dim3(256),
                       0, st, group);
  else
    hipLaunchKernelGGL((dense_join_kernel<MODE, 1>), dim3(unsigned((pieces + 255) / 256), 1, unsigned(count)),
                       dim3(256), 0, st, group);
  return hipGetLastError();
}

template <int LAYOUT, int MODE>
hipError_t launch_mode(const DenseGroup& group, int count, const DensePlan& p, hipStream_t st) {
  constexpr bool DUAL = MODE == kEpiGated || MODE == kEpiKeep;
  const hipError_t err = p.tile == 256   ? launch_shape<DenseShape<LAYOUT, MODE, 256, 256>>(group, count, st)
                         : p.tile == 128 ? launch_shape<DenseShape<LAYOUT, MODE, 128, 128>>(group, count, st)
                         : p.tile == 64  ? launch_shape<DenseShape<LAYOUT, MODE, 64, DUAL ? 128 : 64>>(group, count, st)
                                         : launch_narrow<LAYOUT, MODE>(group, count, st);
  return err != hipSuccess || p.split == 1 ? err : launch_join<MODE>(group, count, st);
}
int64_t part_floats(const DensePlan& p, int64_t M, int N, int dual) {
  return p.split == 1 ? 0 : int64_t(p.split) * (dual ? 2 : 1) * M * ((int64_t(N) + 7) & ~int64_t(7));
}

}  // namespace

size_t dense_part_bytes(int64_t M, int N, int64_t K, int segments, int dual, int count, bool thin) {
  int64_t floats = part_floats(dense_plan(M, N, K, segments, dual, count, false), M, N, dual);
  if (thin && !dual)
    floats = std::max(floats, part_floats(dense_plan(M, N, K, segments, dual, count, true), M, N, dual));
  return size_t(count) * size_t(floats) * sizeof(float);
}

// The most that dense_part_bytes (thin) gives for any M from 1 to this one: the plan
// is the same for 64 rows at a time, and the last of them take the most.
size_t dense_part_most(int64_t M, int N, int64_t K, int segments, int dual, int count) {
  size_t most = 0;
  if ((K + BK - 1) / BK * segments < 4 * kSplits[1]) return 0;
  for (int64_t m = 64;; m += 64) {
    const int64_t at = std::min(m, M);
    if (tiles_of(at, N, dual, kTileCosts[0].tile) * count * kSplits[1] > kSplitGroups) return most;  // nor further on
    most = std::max(most, dense_part_bytes(at, N, K, segments, dual, count, true));
    if (at == M) return most;
  }
}

// At least what dense_part_bytes (not thin) gives for any K up to this one.  A split into u
// parts takes per >= steps / u steps a part, so where the turns of the chip that
// its groups take cost no less, divided by u, than the whole product's, the
// whole product (no join) always costs less.
size_t dense_part_most_deep(int64_t M, int N, int64_t K, int segments, int count) {
  const int64_t steps = (K + BK - 1) / BK * segments;
  int most = 1;
  for (const TileCost& c : kTileCosts) {
    const int64_t tiles = tiles_of(M, N, 0, c.tile) * count, slots = int64_t(256) * c.per_cu;
    if (c.tile == 32) break;
    auto turns = [&](int u) {  // microseconds that a step of every group takes
      const int64_t rest = tiles * u % slots;
      return double(tiles * u / slots) * c.step[c.per_cu - 1] + (rest == 0 ? 0.0 : c.step[rest > 256 ? 1 : 0]);
    };
    for (int u = kSplits[7]; u > most; --u)
      if (steps >= 4 * u && tiles * u <= kSplitGroups && turns(u) < u * turns(1)) most = u;
  }
  return size_t(count) * size_t(part_floats(DensePlan{0, most, 0}, M, N, 0)) * sizeof(float);
}

namespace {

// The plan's part of a product's arguments
void set_plan(DenseArgs& g, const DensePlan& p, float* part) {
  g.split = p.split;
  g.steps_per_split = p.steps;
  g.ld_part = (int64_t(g.N) + 7) & ~int64_t(7);
  g.part = part;
}

}  // namespace

hipError_t launch_dense(const DenseGroup& args, int count, int layout, float* part, hipStream_t st) {
  if (count < 1 || count > kMaxGroup) return hipErrorInvalidValue;
  DenseGroup group = args;
  const DenseArgs& f = group.g[0];
  if (f.M <= 0 || f.N <= 0) return hipSuccess;
  const int mode = f.epi.mode;
  const DensePlan p = dense_plan(f.M, f.N, f.K, f.segments, f.dual, count, narrow(layout, mode));
  if (p.split > 1 && part == nullptr) return hipErrorInvalidValue;
  for (int i = 0; i < count; ++i) {
    DenseArgs& g = group.g[i];
    if (g.segments < 1 || g.segments > kMaxSegments || g.dual != (mode == kEpiGated || mode == kEpiKeep) ||
        g.epi.mode != mode || g.K != f.K || g.segments != f.segments)
      return hipErrorInvalidValue;
    set_plan(g, p, part);
    part += part_floats(p, g.M, g.N, g.dual);
  }
  // the products that the operators are made of
  if (layout == kNT && mode == kEpiOut) return launch_mode<kNT, kEpiOut>(group, count, p, st);
  if (layout == kNT && mode == kEpiGated) return launch_mode<kNT, kEpiGated>(group, count, p, st);
  if (layout == kNT && mode == kEpiKeep) return launch_mode<kNT, kEpiKeep>(group, count, p, st);
  if (layout == kNT && mode == kEpiActBack) return launch_mode<kNT, kEpiActBack>(group, count, p, st);
  if (layout == kNN && mode == kEpiOut) return launch_mode<kNN, kEpiOut>(group, count, p, st);
  if (layout == kNN && mode == kEpiGatedBack) return launch_mode<kNN, kEpiGatedBack>(group, count, p, st);
  if (layout == kTN && mode == kEpiOut) return launch_mode<kTN, kEpiOut>(group, count, p, st);
  return hipErrorInvalidValue;
}

// A layer's gradients of its input (A B) and of its weights (A^T B).  Where both
// take the small tile and fit the chip together they go in one launch: 300 x
// 1024 x 256 in float32 25.1 -> 15.5 us, 512 x 1024 x 1024 in bfloat16 13.0 ->
// 8.2, a feed-forward block of 300 x 1024 x 256 28.6 -> 23.4.  With more
// workgroups than fit it is slower for some (300 x 1024 x 2048 in float32 44.9 ->
// 46.5) and faster for others (512 x 1536 x 1024 in bfloat16 14.7 -> 10.9); those
// are not told apart here and stay in two.
hipError_t launch_dense_gradients(const DenseArgs& data, const DenseGroup& weights, int count, float* part,
                                  hipStream_t st) {
  if (count < 1 || count >= kMaxGroup) return hipErrorInvalidValue;
  typedef DenseShape<kNN, kEpiOut, 64, 64> Data;
  typedef DenseShape<kTN, kEpiOut, 64, 64> Weights;
  static_assert(Data::LDS == Weights::LDS, "one size for both");
  const DenseArgs& w = weights.g[0];
  const DensePlan pd = dense_plan(data.M, data.N, data.K, data.segments, 0, 1, false);
  const DensePlan pw = dense_plan(w.M, w.N, w.K, w.segments, 0, count, false);
  bool together = pd.tile == 64 && pw.tile == 64 && pw.split == 1 && data.epi.mode == kEpiOut && data.dual == 0;
  DenseGroup group{};
  group.g[0] = data;
  set_plan(group.g[0], pd, part);
  int64_t tiles = tiles_of<Data>(data), groups = tiles * pd.split;
  for (int i = 0; i < count; ++i) {
    const DenseArgs& g = weights.g[i];
    together = together && g.epi.mode == kEpiOut && g.dual == 0 && g.K == w.K && g.segments == w.segments;
    group.g[1 + i] = g;
    set_plan(group.g[1 + i], pw, nullptr);
    tiles = std::max(tiles, tiles_of<Weights>(g));
    groups += tiles_of<Weights>(g);
  }
  if (!together || groups > 512) {
    DenseGroup one{};
    one.g[0] = data;
    const hipError_t err = launch_dense(one, 1, kNN, part, st);
    return err != hipSuccess ? err : launch_dense(weights, count, kTN, part, st);
  }
  if (pd.split > 1 && part == nullptr) return hipErrorInvalidValue;
  const hipError_t err = launch_kernel(&dense_pair_kernel<Data, Weights>, Data::LDS, tiles, group, 1 + count, st);
  return err != hipSuccess || pd.split == 1 ? err : launch_join<kEpiOut>(group, 1, st);
}

hipError_t launch_dense_pack(const PackJobs& jobs, int count, bool f32, hipStream_t st) {
  if (count < 0 || count > kMaxPacks) return hipErrorInvalidValue;
  int64_t blocks = 0;
  for (int i = 0; i < count; ++i) blocks = std::max(blocks, (jobs.j[i].rows * (jobs.j[i].ld_dst / 8) + 255) / 256);
  if (blocks == 0) return hipSuccess;
  // (a grid dimension has less than 2^32 threads; past these the blocks go on)
  blocks = std::min(blocks, int64_t(1) << 22);
  if (f32)
    hipLaunchKernelGGL((dense_pack_kernel<float>), dim3(unsigned(blocks), unsigned(count)), dim3(256), 0, st, jobs);
  else
    hipLaunchKernelGGL((dense_pack_kernel<bf16_t>), dim3(unsigned(blocks), unsigned(count)), dim3(256), 0, st, jobs);
  return hipGetLastError();
}

// (a row of sums for each half of a tile's rows, or for each chunk of rows)
size_t dense_sums_bytes(int64_t rows, int cols) {
  return size_t((rows + kSumRows - 1) / kSumRows) * 2 * size_t(cols) * sizeof(float);
}

namespace {

hipError_t join_sums(const float* sums, int64_t n, int cols, void* out, bool f32, hipStream_t st) {
  const dim3 grid((cols + 31) / 32);
  if (f32)
    hipLaunchKernelGGL((dense_colsum_join_kernel<float>), grid, dim3(1024), 0, st, sums, n, cols,
                       static_cast<float*>(out));
  else
    hipLaunchKernelGGL((dense_colsum_join_kernel<bf16_t>), grid, dim3(1024), 0, st, sums, n, cols,
                       static_cast<bf16_t*>(out));
  return hipGetLastError();
}

}  // namespace

hipError_t launch_dense_colsum(const void* src, bool src_f32, int64_t ld, int64_t rows, int cols, void* out, bool f32,
                               float* sums, hipStream_t st) {
  const int64_t chunks = (rows + kSumRows - 1) / kSumRows;
  // chunks lie along x: there are up to 2^18 of them
  const dim3 grid(unsigned(chunks), (cols + 255) / 256);
  if (src_f32)
    hipLaunchKernelGGL((dense_colsum_kernel<float>), grid, dim3(256), 0, st, static_cast<const float*>(src), ld, rows,
                       cols, sums);
  else
    hipLaunchKernelGGL((dense_colsum_kernel<bf16_t>), grid, dim3(256), 0, st, static_cast<const bf16_t*>(src), ld, rows,
                       cols, sums);
  const hipError_t err = hipGetLastError();
  return err != hipSuccess ? err : join_sums(sums, chunks, cols, out, f32, st);
}

hipError_t launch_dense_act_back(const DenseArgs& args, void* dbias, float* sums, float* part, hipStream_t st) {
  DenseGroup group{};
  DenseArgs& g = group.g[0];
  g = args;
  if (dbias != nullptr) g.epi.sums = sums;
  hipError_t err = launch_dense(group, 1, kNT, part, st);
  if (err != hipSuccess || dbias == nullptr) return err;
  const DensePlan p = dense_plan(g.M, g.N, g.K, g.segments, 0, 1, false);
  if (p.split > 1) {
    set_plan(g, p, part);
    return launch_dense_colsum(part, true, g.ld_part, g.M, g.N, dbias, g.epi.f32, sums, st);
  }
  const int64_t rows = std::max(p.tile, 64);
  return join_sums(sums, (g.M + rows - 1) / rows * 2, g.N, dbias, g.epi.f32, st);
}

}  // namespace moe
