// Norms after a block and before the next one, fused with the gate and the
// residual stream between them.
//
//   p = unit(f), n = p w_post + b_post, u = s r + gate n, q = unit(u),
//   h = q w_pre + b_pre, unit(v) = (v - m) / sqrt(mean((v - m)^2) + eps)
// with m the row's mean (layer norm) or 0 (RMS norm), r the residual stream
// and f the block's output.  All in float32, rounded once at each store; the
// mean is taken out before the squares are summed, so a row far from zero
// loses nothing.
//
// Backward of <du, u> + <dh, h>, from r and f again (nothing is kept from the
// forward):
//   a = dh w_pre, e = du + (a - [mean a] - q mean(a q)) / sigma_u, dr = s e,
//   dgate = sum e n, g = e gate, dw_post = sum g p, db_post = sum g,
//   c = g w_post, df = (c - [mean c] - p mean(c p)) / sigma_f,
//   dw_pre = sum dh q, db_pre = sum dh
// ([.] for the layer norm).
//
// Memory-bound: 4 (forward) or 6 (backward) rows move per token and about 14
// or 40 operations an element.  A row therefore stays in registers from its
// load to its stores, vectors of 8 consecutive elements a thread, so every
// element is read and written once however many statistics the row needs.  A
// row of up to 1024 is one wave's, and needs no barrier; a longer row is one
// workgroup's, of up to 512 threads with two vectors each (past 8192 four).
// A worker (that wave or workgroup) takes a contiguous range of rows: it keeps
// the norm weights in registers over them, has its next row's loads in flight
// while it works on the present one, and in the backward adds its columns'
// weight gradients up in registers, one partial row a workgroup, which a
// second kernel joins in workgroup order (deterministic, no atomics).  Where
// the backward's registers are short (layer norm, float32, ragged and wide
// rows), the weights are read again for every row, from the caches, and past
// 8192 the next row is not fetched ahead: 4096 rows of 7168 with a layer norm
// 340 -> 127 us, 2048 of 16384 with an RMS norm 722 -> 174 us.  That is not
// enough everywhere: of float32 past 1024 the backward's layer norm and ragged
// RMS norm put 5 to 61 registers out to memory, every backward past 8192 63 to
// 248, and there the forward of float32 36 (ragged) to 174 (layer norm).
//
// Measured: forward, 8192 rows of 7168 in bfloat16, 96 us = 4.9 TB/s, what a
// large copy reaches on this card (5.0), as a layer norm 99, float32 191 either
// way, without gate and first norm 95; one row 4 us, a launch's latency.
// Backward, 4096 rows of 7168 in bfloat16, RMS: 80 us = 4.4 TB/s and 6 us for
// the join; as a layer norm 127 us (six rounds of sums a row and the parameters
// again, several times a row), float32 174 and 235.  2048 rows of 16384: forward
// 57, float32 layer norm 189; backward 174, as a layer norm 460, float32 476, all
// by the registers put out.  777 rows of 1001 in float32, layer norm: 11 + 4.5
// us, the time that one wave takes for its row or two.  Of the backward's 80 us
// the sums' barriers and the column gradients' arithmetic are what is above the
// copy's 70.
#include "block.h"

namespace moe {

namespace {

// Sums over a row's threads, in a fixed order, every thread gets them.  Lane
// moves by DPP leave each 16-lane row's sum in its lanes; one wave alone adds
// its four.  Several waves leave their rows' sums in LDS (up to 64), and behind
// one barrier every wave adds those up the same way.  Two alternating LDS slots
// are enough: a wave writes a slot again only after the barrier of the sum
// between, which every wave reaches after its reads of that slot.
struct RowSum {
  float* lds;  // [2][5][64]
  int nrow;    // 16-lane rows of the workgroup
  int turn;
  static MOE_DEV float lanes16(float v) {
    v = add_dpp<0xb1>(v);   // lane ^ 1
    v = add_dpp<0x4e>(v);   // lane ^ 2
    v = add_dpp<0x124>(v);  // row_ror:4
    return add_dpp<0x128>(v);
  }
  static MOE_DEV float four_rows(float v) {
    float s = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), 0));
#pragma unroll
    for (int r = 16; r < 64; r += 16) s += __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), r));
    return s;
  }
  template <bool ONE_WAVE, int N> MOE_DEV void sums(float (&v)[N]) {
    static_assert(N <= 5, "LDS slots");
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = lanes16(v[i]);
    if (!ONE_WAVE) {
      float* s = lds + turn * 320;
      turn ^= 1;
      if ((threadIdx.x & 15) == 0) {
#pragma unroll
        for (int i = 0; i < N; ++i) s[i * 64 + (threadIdx.x >> 4)] = v[i];
      }
      __syncthreads();
      const int lane = threadIdx.x & 63;
#pragma unroll
      for (int i = 0; i < N; ++i) v[i] = lanes16(lane < nrow ? s[i * 64 + lane] : 0.f);
    }
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = four_rows(v[i]);
  }
  template <bool ONE_WAVE> MOE_DEV float sum(float v) {
    float a[1] = {v};
    sums<ONE_WAVE, 1>(a);
    return a[0];
  }
};

// Which elements of a row a thread has, vector j, i = 0 .. 7.  WHOLE (the row's
// length is a multiple of 8): eight in a row, one 16-byte access (two for
// float32), all inside the row or all past it.  Else one from each of eight
// pieces of the row, each piece read in full by the threads together.
template <bool WHOLE> struct Cols {
  int tid, nthr, H;
  MOE_DEV int at(int j, int i) const { return WHOLE ? (j * nthr + tid) * 8 + i : (j * 8 + i) * nthr + tid; }
  MOE_DEV bool in(int j, int i) const { return at(j, i) < H; }
};

// A row in memory is accessed as a buffer of the row's extent: what lies past
// its end reads as zero and is not written, with no comparison, and a row costs
// two scalar registers instead of addresses in every lane.
template <typename TE> MOE_DEV __amdgpu_buffer_rsrc_t row_rsrc(const TE* row, int H) {
  return buffer_rsrc(row, uint32_t(H) * uint32_t(sizeof(TE)));
}

// raw (unconverted) elements of a row, so that a row in flight costs its own
// bytes in registers
template <typename TE, bool WHOLE> struct Raw8;
template <bool WHOLE> struct Raw8<bf16_t, WHOLE> {
  typedef bf16_t TE;
  u32x4 a;
  MOE_DEV void load(const bf16_t* row, const Cols<WHOLE>& c, int j) {
    if (WHOLE) {
      a = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(row_rsrc(row, c.H), c.at(j, 0) * 2, 0, 0));
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t lo = __builtin_amdgcn_raw_buffer_load_b16(row_rsrc(row, c.H), c.at(j, 2 * i) * 2, 0, 0);
        const uint32_t hi = __builtin_amdgcn_raw_buffer_load_b16(row_rsrc(row, c.H), c.at(j, 2 * i + 1) * 2, 0, 0);
        a[i] = lo | (hi << 16);
      }
    }
  }
  MOE_DEV void fill(bool one) { a = u32x4{1u, 1u, 1u, 1u} * (one ? 0x3f803f80u : 0u); }
  // what is made of the value is made anew behind this point: without it the
  // float32 forms of a row's parameters, twice as many registers, are kept
  // over the worker's rows in place of the packed ones
  MOE_DEV void pin() { asm volatile("" : "+v"(a)); }
  MOE_DEV void get(float (&v)[8]) const { unpack8(a, v); }
};
template <bool WHOLE> struct Raw8<float, WHOLE> {
  typedef float TE;
  float a[8];
  MOE_DEV void load(const float* row, const Cols<WHOLE>& c, int j) {
    if (WHOLE) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const f32x4 x = __builtin_bit_cast(
            f32x4, __builtin_amdgcn_raw_buffer_load_b128(row_rsrc(row, c.H), c.at(j, 4 * h) * 4, 0, 0));
#pragma unroll
        for (int i = 0; i < 4; ++i) a[4 * h + i] = x[i];
      }
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        a[i] = __int_as_float(__builtin_amdgcn_raw_buffer_load_b32(row_rsrc(row, c.H), c.at(j, i) * 4, 0, 0));
    }
  }
  MOE_DEV void fill(bool one) {
#pragma unroll
    for (int i = 0; i < 8; ++i) a[i] = one ? 1.f : 0.f;
  }
  MOE_DEV void pin() {}
  MOE_DEV void get(float (&v)[8]) const {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = a[i];
  }
};
typedef uint32_t u32x4_raw __attribute__((__vector_size__(16)));
template <bool WHOLE, typename TO> MOE_DEV void put(TO* row, const Cols<WHOLE>& c, int j, const float (&v)[8]) {
  if (!WHOLE) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if (sizeof(TO) == 2)
        __builtin_amdgcn_raw_buffer_store_b16(f32_to_bf16(v[i]), row_rsrc(row, c.H), c.at(j, i) * 2, 0, 0);
      else
        __builtin_amdgcn_raw_buffer_store_b32(__float_as_int(v[i]), row_rsrc(row, c.H), c.at(j, i) * 4, 0, 0);
    }
  } else if (sizeof(TO) == 2) {
    __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4_raw, pack8(v)), row_rsrc(row, c.H), c.at(j, 0) * 2,
                                           0, 0);
  } else {
#pragma unroll
    for (int h = 0; h < 2; ++h)
      __builtin_amdgcn_raw_buffer_store_b128(
          __builtin_bit_cast(u32x4_raw, f32x4{v[4 * h], v[4 * h + 1], v[4 * h + 2], v[4 * h + 3]}),
          row_rsrc(row, c.H), c.at(j, 4 * h) * 4, 0, 0);
  }
}

// v becomes the unit row (0 past the row's end); returns 1 / sigma
template <class S>
MOE_DEV float unit_row(float (&v)[S::NV][8], const Cols<S::WHOLE>& c, float eps, RowSum& rs) {
  constexpr int NV = S::NV;
  const float rh = 1.0f / float(c.H);
  if (S::LAYER) {
    float s = 0.f;
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
      for (int i = 0; i < 8; ++i) s += v[j][i];
    const float m = rs.sum<S::ONE_WAVE>(s) * rh;
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
      for (int i = 0; i < 8; ++i) v[j][i] = c.in(j, i) ? v[j][i] - m : 0.f;
  }
  float ss = 0.f;
#pragma unroll
  for (int j = 0; j < NV; ++j)
#pragma unroll
    for (int i = 0; i < 8; ++i) ss = fmaf(v[j][i], v[j][i], ss);
  const float inv = 1.0f / sqrtf(rs.sum<S::ONE_WAVE>(ss) * rh + eps);
#pragma unroll
  for (int j = 0; j < NV; ++j)
#pragma unroll
    for (int i = 0; i < 8; ++i) v[j][i] *= inv;
  return inv;
}

template <class R, class C> MOE_DEV void take(R& r, const void* p, const C& c, int j, bool one) {
  if (p) r.load(static_cast<const typename R::TE*>(p), c, j);
  else r.fill(one);
}

// v w, or v w + b
template <class S, class R> MOE_DEV void affine(float (&v)[8], const R& weight, const R& bias) {
  float w[8], b[8];
  weight.get(w);
  if (S::LAYER) bias.get(b);
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = S::LAYER ? fmaf(v[i], w[i], b[i]) : v[i] * w[i];
}

// first row of worker w of n over T rows
MOE_DEV int64_t worker_row(int64_t T, int w, int n) { return T * w / n; }

// NV: vectors of 8 a thread; LAYER: layer norm; WHOLE: H % 8 == 0
template <typename TE_, int NV_, bool ONE_WAVE_, bool LAYER_, bool WHOLE_> struct NormShape {
  typedef TE_ TE;
  static constexpr int NV = NV_;
  static constexpr bool ONE_WAVE = ONE_WAVE_, LAYER = LAYER_, WHOLE = WHOLE_;
  // backward: the parameters are read again for every row (from the caches)
  // where keeping them would put (more) other registers out to memory
  static constexpr bool REREAD = !ONE_WAVE && (LAYER || !WHOLE || NV > 2 || sizeof(TE) == 4);
  // ... and the next row is not kept in flight
  static constexpr bool FETCH_AHEAD = NV <= 2;
};

// NormArgs::options, set by the launchers from the pointers given
constexpr int kNormPost = 1, kNormGate = 2, kNormU = 4, kNormPre = 8, kNormDResidual = 16, kNormDBranch = 32;

int norm_options(const NormArgs& a) {
  return (a.branch && a.w_post ? kNormPost : 0) | (a.gate_rows ? kNormGate : 0) | (a.u ? kNormU : 0) |
         (a.h || a.dh ? kNormPre : 0) | (a.d_residual ? kNormDResidual : 0) | (a.d_branch ? kNormDBranch : 0);
}

constexpr int kRowThreads = 512;  // most threads of a workgroup that shares a row
constexpr int kRowWaves = 4;  // waves (one row each) of a workgroup of one-wave workers

}  // namespace

// ---------------------------------------------------------------- forward

template <class S>
__global__ __launch_bounds__(S::ONE_WAVE ? 64 * kRowWaves : kRowThreads) void norm_forward_kernel(NormArgs a) {
  typedef typename S::TE TE;
  constexpr int NV = S::NV;
  constexpr bool ONE = S::ONE_WAVE;
  __shared__ float lds[640];
  const int H = a.H;
  const int tid = ONE ? threadIdx.x & 63 : threadIdx.x;
  const int nthr = ONE ? 64 : blockDim.x;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int worker = ONE ? blockIdx.x * kRowWaves + wave : blockIdx.x;
  if (worker >= a.workers) return;  // whole waves, and no barrier below for them
  RowSum rs{lds, int(blockDim.x >> 4), 0};
  const Cols<S::WHOLE> c{tid, nthr, H};

  const TE* r = static_cast<const TE*>(a.residual);
  const TE* f = static_cast<const TE*>(a.branch);
  // absent parameters are ones or zeros: the arithmetic is the same
  typedef Raw8<TE, S::WHOLE> Raw;
  Raw wpost[NV], wpre[NV], gate[NV], bpost[S::LAYER ? NV : 1], bpre[S::LAYER ? NV : 1];
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    take(wpost[j], a.w_post, c, j, true);
    take(wpre[j], a.w_pre, c, j, true);
    gate[j].fill(true);
    if (S::LAYER) {
      take(bpost[j], a.b_post, c, j, false);
      take(bpre[j], a.b_pre, c, j, false);
    }
  }
  const int64_t t0 = worker_row(a.T, worker, a.workers), t1 = worker_row(a.T, worker + 1, a.workers);
  int64_t group_end = t0;
  Raw rn[NV], fn[NV];
  r += t0 * a.ld_residual;
  if (f) f += t0 * a.ld_branch;
  TE* u_row = static_cast<TE*>(a.u) + (a.u ? t0 * a.ld_u : 0);
  TE* h_row = static_cast<TE*>(a.h) + (a.h ? t0 * a.ld_h : 0);
  auto fetch = [&]() {  // the next row
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      rn[j].load(r, c, j);
      if (f) fn[j].load(f, c, j);
      else fn[j].fill(false);
    }
    r += a.ld_residual;
    if (f) f += a.ld_branch;
  };
  if (t0 < t1) fetch();
  for (int64_t t = t0; t < t1; ++t) {
    // The options are read anew for every row: the loop is not to be cloned
    // for each combination of them.
    int opt = a.options;
    asm volatile("" : "+s"(opt));
    if ((opt & kNormGate) && t >= group_end) {
      const int64_t group = t / a.gate_rows;
      group_end = (group + 1) * a.gate_rows;
#pragma unroll
      for (int j = 0; j < NV; ++j) gate[j].load(static_cast<const TE*>(a.gate) + group * H, c, j);
    }
    float u[NV][8], v[NV][8];
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      rn[j].get(u[j]);
      fn[j].get(v[j]);
      wpost[j].pin();
      wpre[j].pin();
      gate[j].pin();
    }
    if (t + 1 < t1) fetch();
    if (opt & kNormPost) {
      unit_row<S>(v, c, a.eps, rs);
#pragma unroll
      for (int j = 0; j < NV; ++j) affine<S>(v[j], wpost[j], bpost[S::LAYER ? j : 0]);
    }
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      float g[8];
      gate[j].get(g);
#pragma unroll
      for (int i = 0; i < 8; ++i) u[j][i] = fmaf(v[j][i], g[i], a.scale * u[j][i]);
      if (opt & kNormU) put(u_row, c, j, u[j]);
    }
    if (opt & kNormPre) {
      unit_row<S>(u, c, a.eps, rs);
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        affine<S>(u[j], wpre[j], bpre[S::LAYER ? j : 0]);
        put(h_row, c, j, u[j]);
      }
    }
    if (a.u) u_row += a.ld_u;
    if (a.h) h_row += a.ld_h;
  }
}

// ---------------------------------------------------------------- backward

// The gate row's gradient goes straight to its place where the worker has all
// of the row's tokens.  A gate row that several workers share is joined from
// their partial rows: gpart[2 w] is worker w's share of a row begun before its
// range, gpart[2 w + 1] of one begun inside it and going on after it.
template <class S>
__global__ __launch_bounds__(S::ONE_WAVE ? 64 * kRowWaves : kRowThreads) void norm_backward_kernel(NormArgs a) {
  typedef typename S::TE TE;
  constexpr int NV = S::NV;
  constexpr bool ONE = S::ONE_WAVE;
  // sums of a row in progress, or of the workers of a workgroup at the end
  __shared__ float lds[ONE ? kRowWaves * 64 * 8 * NV : 640];
  const int H = a.H;
  const float rh = 1.0f / float(H);
  const int tid = ONE ? threadIdx.x & 63 : threadIdx.x;
  const int nthr = ONE ? 64 : blockDim.x;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int worker = ONE ? blockIdx.x * kRowWaves + wave : blockIdx.x;
  RowSum rs{lds, int(blockDim.x >> 4), 0};
  const Cols<S::WHOLE> c{tid, nthr, H};

  const TE* r = static_cast<const TE*>(a.residual);
  const TE* f = static_cast<const TE*>(a.branch);
  const TE* du = static_cast<const TE*>(a.du);
  const TE* dh = static_cast<const TE*>(a.dh);
  typedef Raw8<TE, S::WHOLE> Raw;
  constexpr int NB = S::LAYER ? NV : 1;  // vectors of what only the layer norm has
  constexpr int NP = S::REREAD ? 1 : NV;
  Raw wpost_[NP], wpre_[NP], gate_[NP], bpost_[S::REREAD ? 1 : NB];
  float swpost[NV][8], swpre[NV][8], sgate[NV][8], sbpost[NB][8], sbpre[NB][8];
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    if (!S::REREAD) {
      take(wpost_[j], a.w_post, c, j, true);
      take(wpre_[j], a.w_pre, c, j, true);
      gate_[j].fill(true);
      if (S::LAYER) take(bpost_[j], a.b_post, c, j, false);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      swpost[j][i] = swpre[j][i] = sgate[j][i] = 0.f;
      if (S::LAYER) sbpost[j][i] = sbpre[j][i] = 0.f;
    }
  }

  // (workers past the last have no rows, and join the others at the end)
  const int64_t t0 = worker_row(a.T, min(worker, a.workers), a.workers);
  const int64_t t1 = worker_row(a.T, min(worker + 1, a.workers), a.workers);
  int64_t group = -1, group_end = t0;
  auto read_again = [&](const void* p, int j, bool one) __attribute__((always_inline)) {
    Raw r;
    take(r, p, c, j, one);
    return r;
  };
  auto wpost = [&](int j) __attribute__((always_inline)) { return S::REREAD ? read_again(a.w_post, j, true) : wpost_[S::REREAD ? 0 : j]; };
  auto wpre = [&](int j) __attribute__((always_inline)) { return S::REREAD ? read_again(a.w_pre, j, true) : wpre_[S::REREAD ? 0 : j]; };
  auto bpost = [&](int j) __attribute__((always_inline)) { return S::REREAD ? read_again(a.b_post, j, false) : bpost_[S::REREAD ? 0 : j]; };
  auto gate = [&](int j) __attribute__((always_inline)) {
    return S::REREAD ? read_again(a.gate ? static_cast<const TE*>(a.gate) + group * H : nullptr, j, true)
                     : gate_[S::REREAD ? 0 : j];
  };
  // the gate row `group` ends at row `end` of the worker's range
  auto flush_gate = [&](int64_t end) {
    if (a.dgate == nullptr || group < 0) return;
    const int64_t first = group * a.gate_rows, last = first + a.gate_rows;
    const bool whole = first >= t0 && last <= end;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      if (whole) put(static_cast<TE*>(a.dgate) + group * H, c, j, sgate[j]);
      else put(a.gpart + (2 * int64_t(worker) + (first >= t0 ? 1 : 0)) * H, c, j, sgate[j]);
#pragma unroll
      for (int i = 0; i < 8; ++i) sgate[j][i] = 0.f;
    }
  };
  Raw rn[NV], fn[NV], dun[NV], dhn[NV];
  r += t0 * a.ld_residual;
  if (f) f += t0 * a.ld_branch;
  if (du) du += t0 * a.ld_du;
  if (dh) dh += t0 * a.ld_dh;
  TE* dr_row = static_cast<TE*>(a.d_residual) + (a.d_residual ? t0 * a.ld_dr : 0);
  TE* db_row = static_cast<TE*>(a.d_branch) + (a.d_branch ? t0 * a.ld_db : 0);
  auto fetch = [&]() {  // the next row
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      rn[j].load(r, c, j);
      if (f) fn[j].load(f, c, j);
      else fn[j].fill(false);
      if (du) dun[j].load(du, c, j);
      else dun[j].fill(false);
      if (dh) dhn[j].load(dh, c, j);
      else dhn[j].fill(false);
    }
    r += a.ld_residual;
    if (f) f += a.ld_branch;
    if (du) du += a.ld_du;
    if (dh) dh += a.ld_dh;
  };
  if (S::FETCH_AHEAD && t0 < t1) fetch();
  for (int64_t t = t0; t < t1; ++t) {
    int opt = a.options;  // read anew for every row, as in the forward
    asm volatile("" : "+s"(opt));
    if ((opt & kNormGate) && t >= group_end) {
      flush_gate(t);
      group = t / a.gate_rows;
      group_end = (group + 1) * a.gate_rows;
#pragma unroll
      for (int j = 0; j < NV && !S::REREAD; ++j) gate_[j].load(static_cast<const TE*>(a.gate) + group * H, c, j);
    }
    if (!S::FETCH_AHEAD) fetch();
    float q[NV][8], p[NV][8], e[NV][8], d[NV][8];  // u, then q; p; du, then e; dh, then a
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      rn[j].get(q[j]);
      fn[j].get(p[j]);
      dun[j].get(e[j]);
      dhn[j].get(d[j]);
      if (!S::REREAD) {
        wpost_[j].pin();
        wpre_[j].pin();
        gate_[j].pin();
      }
    }
    if (S::FETCH_AHEAD && t + 1 < t1) fetch();
    float inv_f = 1.f;
    if (opt & kNormPost) inv_f = unit_row<S>(p, c, a.eps, rs);
    float s3 = 0.f, s4 = 0.f;  // row means of c and c p
    if (!S::LAYER) {
      // Everything that the rest of the row needs from its other threads in one
      // round of sums: with k = mean(a u) / sigma_u^2, e = du + (a - k u) / sigma_u,
      // and c p = e (gate n) is linear in du, a and u.
      float m[5] = {0.f, 0.f, 0.f, 0.f, 0.f};  // u u, a u, and gate n with du, a, u
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        float w[8], g[8], x[8];
        wpost(j).get(w);
        gate(j).get(g);
        wpre(j).get(x);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float ng = p[j][i] * w[i] * g[i], aw = d[j][i] * x[i];
          q[j][i] = fmaf(a.scale, q[j][i], ng);
          m[0] = fmaf(q[j][i], q[j][i], m[0]);
          m[1] = fmaf(aw, q[j][i], m[1]);
          m[2] = fmaf(ng, e[j][i], m[2]);
          m[3] = fmaf(ng, aw, m[3]);
          m[4] = fmaf(ng, q[j][i], m[4]);
        }
      }
      rs.template sums<ONE, 5>(m);
      s4 = m[2] * rh;
      if (opt & kNormPre) {
        const float inv_u = 1.0f / sqrtf(m[0] * rh + a.eps), k = inv_u * inv_u * (m[1] * rh);
        s4 = fmaf(inv_u, (m[3] - k * m[4]) * rh, s4);
#pragma unroll
        for (int j = 0; j < NV; ++j) {
          float x[8];
          wpre(j).get(x);
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            swpre[j][i] = fmaf(d[j][i] * inv_u, q[j][i], swpre[j][i]);
            e[j][i] = fmaf(inv_u, fmaf(-k, q[j][i], d[j][i] * x[i]), e[j][i]);
          }
        }
      }
    } else {
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        float n[8], g[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) n[i] = p[j][i];
        affine<S>(n, wpost(j), bpost(S::LAYER ? j : 0));
        gate(j).get(g);
#pragma unroll
        for (int i = 0; i < 8; ++i) q[j][i] = fmaf(n[i], g[i], a.scale * q[j][i]);
      }
      if (opt & kNormPre) {
        const float inv_u = unit_row<S>(q, c, a.eps, rs);
        float m[2] = {0.f, 0.f};
#pragma unroll
        for (int j = 0; j < NV; ++j) {
          float w[8];
          wpre(j).get(w);
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            swpre[j][i] = fmaf(d[j][i], q[j][i], swpre[j][i]);
            if (S::LAYER) sbpre[S::LAYER ? j : 0][i] += d[j][i];
            d[j][i] *= w[i];
            m[0] += d[j][i];
            m[1] = fmaf(d[j][i], q[j][i], m[1]);
          }
        }
        rs.template sums<ONE, 2>(m);
#pragma unroll
        for (int j = 0; j < NV; ++j)
#pragma unroll
          for (int i = 0; i < 8; ++i) e[j][i] = fmaf(inv_u, d[j][i] - m[0] * rh - q[j][i] * (m[1] * rh), e[j][i]);
      }
    }
    // e is the gradient at u
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      float w[8], g[8], n[8];
      if (opt & kNormDResidual) {
#pragma unroll
        for (int i = 0; i < 8; ++i) n[i] = a.scale * e[j][i];
        put(dr_row, c, j, n);
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) n[i] = p[j][i];
      affine<S>(n, wpost(j), bpost(S::LAYER ? j : 0));
      gate(j).get(g);
      wpost(j).get(w);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        sgate[j][i] = fmaf(e[j][i], n[i], sgate[j][i]);
        e[j][i] *= g[i];
        swpost[j][i] = fmaf(e[j][i], p[j][i], swpost[j][i]);
        if (S::LAYER) sbpost[S::LAYER ? j : 0][i] += e[j][i];
        e[j][i] *= w[i];
        if (S::LAYER) {
          s3 += e[j][i];
          s4 = fmaf(e[j][i], p[j][i], s4);
        }
      }
    }
    if (opt & kNormDResidual) dr_row += a.ld_dr;
    if (!(opt & kNormDBranch)) continue;
    if (opt & kNormPost) {
      if (S::LAYER) {
        float m[2] = {s3, s4};
        rs.template sums<ONE, 2>(m);
        s3 = m[0] * rh;
        s4 = m[1] * rh;
      }
#pragma unroll
      for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int i = 0; i < 8; ++i) e[j][i] = inv_f * (e[j][i] - s3 - p[j][i] * s4);
    }
#pragma unroll
    for (int j = 0; j < NV; ++j) put(db_row, c, j, e[j]);
    db_row += a.ld_db;
  }
  flush_gate(t1);
  const int64_t plane = int64_t(gridDim.x) * H;
  float* part = a.part + int64_t(blockIdx.x) * H;
  // one partial row a workgroup: of its one worker, or of its four in worker order
  auto leave = [&](float (&v)[NV][8], float* row) __attribute__((always_inline)) {
    if (!ONE) {
#pragma unroll
      for (int j = 0; j < NV; ++j) put(row, c, j, v[j]);
      return;
    }
    constexpr int W = 64 * 8 * NV;  // columns that a wave covers
    __syncthreads();
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
      for (int i = 0; i < 8; ++i) lds[(threadIdx.x >> 6) * W + c.at(j, i)] = v[j][i];
    __syncthreads();
    for (int col = threadIdx.x; col < H; col += 64 * kRowWaves) {
      float t = lds[col];
#pragma unroll
      for (int w = 1; w < kRowWaves; ++w) t += lds[w * W + col];
      row[col] = t;
    }
  };
  if (a.dw_post) leave(swpost, part);
  if (a.dw_pre) leave(swpre, part + 2 * plane);
  if constexpr (S::LAYER) {
    if (a.db_post) leave(sbpost, part + plane);
    if (a.db_pre) leave(sbpre, part + 3 * plane);
  }
}

// Worker of row t: the largest w with T w / workers <= t
MOE_DEV int64_t row_worker(const NormArgs& a, int64_t t) { return ((t + 1) * a.workers - 1) / a.T; }

// Joins the workgroups' partial rows in their order: blockIdx.y 0..3 the weight
// gradients, 4 + g the gate row g.  A workgroup has 64 columns and 16 shares of
// the rows (share k: rows k, k + 16, ...), added up share by share.
constexpr int kJoinShares = 16;
template <typename TE>
__global__ __launch_bounds__(64 * kJoinShares) void norm_join_kernel(NormArgs a) {
  __shared__ float acc[kJoinShares][64];
  const int lane = threadIdx.x & 63, share = threadIdx.x >> 6;
  const int col = blockIdx.x * 64 + lane;
  const int which = blockIdx.y;
  TE* out;
  const float* src;
  int64_t first, last, step;
  if (which < 4) {
    void* const outs[4] = {a.dw_post, a.db_post, a.dw_pre, a.db_pre};
    out = static_cast<TE*>(outs[which]);
    src = a.part + which * a.partials * int64_t(a.H);
    first = 0;
    last = a.partials;
    step = a.H;
  } else {
    const int64_t g = which - 4;
    first = row_worker(a, g * a.gate_rows);
    last = row_worker(a, (g + 1) * a.gate_rows - 1) + 1;
    if (last - first == 1) return;  // one worker had the whole row and wrote it
    out = static_cast<TE*>(a.dgate) + g * a.H;
    src = a.gpart;
    step = 2 * int64_t(a.H);
  }
  if (out == nullptr) return;
  float s = 0.f;
  if (col < a.H) {
#pragma unroll 8
    for (int64_t w = first + share; w < last; w += kJoinShares)
      s += src[w * step + (which >= 4 && w == first ? a.H : 0) + col];
  }
  acc[share][lane] = s;
  __syncthreads();
  if (share == 0 && col < a.H) {
    s = 0.f;
#pragma unroll
    for (int k = 0; k < kJoinShares; ++k) s += acc[k][lane];
    out[col] = from_f32<TE>(s);
  }
}

// The same for gate rows where there are many of them, each shared by a few
// workers: blockIdx.y is worker b, for the gate row that began in its range and
// goes on past it, if there is one.
constexpr int kFewGates = 64;  // up to here the join above takes them
template <typename TE> __global__ __launch_bounds__(256) void norm_gate_join_kernel(NormArgs a) {
  const int col = blockIdx.x * 256 + threadIdx.x;
  const int64_t b = blockIdx.y, end = worker_row(a.T, int(b) + 1, a.workers);
  const int64_t g = end / a.gate_rows, r0 = g * a.gate_rows;
  if (r0 == end || r0 < worker_row(a.T, int(b), a.workers) || col >= a.H) return;
  const int64_t last = row_worker(a, r0 + a.gate_rows - 1);
  float s = a.gpart[(2 * b + 1) * a.H + col];
  for (int64_t w = b + 1; w <= last; ++w) s += a.gpart[2 * w * a.H + col];
  (static_cast<TE*>(a.dgate) + g * a.H)[col] = from_f32<TE>(s);
}

// ---------------------------------------------------------------- launches

namespace {

struct NormPlan {
  bool one_wave;
  int nv, threads;  // of a workgroup
};
NormPlan norm_plan(int H) {
  if (H <= 1024) return {true, H <= 512 ? 1 : 2, 64 * kRowWaves};
  const int nv = H <= 2 * 8 * kRowThreads ? 2 : 4;
  return {false, nv, ((H + 8 * nv - 1) / (8 * nv) + 63) / 64 * 64};
}
static_assert(4 * 8 * kRowThreads >= kNormMaxHidden, "the widest row fits a workgroup");

// F::launch<NormShape<...>> for the shape, kind and alignment of the call
template <class F, typename TE, int NV, bool ONE> void pick_form(const NormArgs& a, const F& f) {
  const bool whole = a.H % 8 == 0;
  if (a.layer && whole) f(NormShape<TE, NV, ONE, true, true>{});
  else if (a.layer) f(NormShape<TE, NV, ONE, true, false>{});
  else if (whole) f(NormShape<TE, NV, ONE, false, true>{});
  else f(NormShape<TE, NV, ONE, false, false>{});
}
template <class F, typename TE> void pick_shape(const NormArgs& a, const NormPlan& p, const F& f) {
  if (p.one_wave && p.nv == 1) pick_form<F, TE, 1, true>(a, f);
  else if (p.one_wave) pick_form<F, TE, 2, true>(a, f);
  else if (p.nv == 2) pick_form<F, TE, 2, false>(a, f);
  else pick_form<F, TE, 4, false>(a, f);
}

template <typename TE>
hipError_t launch_forward(const NormArgs& a, const NormPlan& p, unsigned grid, hipStream_t st) {
  auto f = [&](auto shape) {
    hipLaunchKernelGGL((norm_forward_kernel<decltype(shape)>), dim3(grid), dim3(p.threads), 0, st, a);
  };
  pick_shape<decltype(f), TE>(a, p, f);
  return hipGetLastError();
}

template <typename TE>
hipError_t launch_backward(const NormArgs& a, const NormPlan& p, unsigned grid, hipStream_t st) {
  auto f = [&](auto shape) {
    hipLaunchKernelGGL((norm_backward_kernel<decltype(shape)>), dim3(grid), dim3(p.threads), 0, st, a);
  };
  pick_shape<decltype(f), TE>(a, p, f);
  const hipError_t err = hipGetLastError();
  if (err != hipSuccess) return err;
  NormArgs join = a;
  join.partials = int(grid);
  const int64_t gates = a.dgate ? a.T / a.gate_rows : 0;
  const unsigned jobs = 4 + unsigned(gates <= kFewGates ? gates : 0);
  hipLaunchKernelGGL((norm_join_kernel<TE>), dim3((a.H + 63) / 64, jobs), dim3(64 * kJoinShares), 0, st, join);
  // (a gate row of one token is one worker's, and a lone worker has them all)
  if (gates > kFewGates && a.gate_rows > 1 && a.workers > 1)
    hipLaunchKernelGGL((norm_gate_join_kernel<TE>), dim3((a.H + 255) / 256, a.workers - 1), dim3(256), 0, st, join);
  return hipGetLastError();
}

}  // namespace

// Workers of the backward: enough for every CU, few enough that their partial
// rows stay small beside the tokens' own rows.
int norm_backward_workers(int64_t T, int H) {
  const NormPlan p = norm_plan(H);
  const int64_t most = p.one_wave ? (p.nv == 1 ? 2048 : 1024) : int64_t(256) * std::max(1, 512 / p.threads);
  return int(T < most ? T : most);
}

hipError_t launch_norm_forward(const NormArgs& args, bool bf16, hipStream_t st) {
  NormArgs a = args;
  a.options = norm_options(a);
  const NormPlan p = norm_plan(a.H);
  // every wave slot of the chip: workers hold their weights over their rows
  const int64_t most = p.one_wave ? 256 * 32 : 256 * (2048 / p.threads);
  a.workers = int(a.T < most ? a.T : most);
  const unsigned grid = unsigned(p.one_wave ? (a.workers + kRowWaves - 1) / kRowWaves : a.workers);
  return bf16 ? launch_forward<bf16_t>(a, p, grid, st) : launch_forward<float>(a, p, grid, st);
}

hipError_t launch_norm_backward(const NormArgs& args, bool bf16, hipStream_t st) {
  NormArgs a = args;
  a.options = norm_options(a);
  const NormPlan p = norm_plan(a.H);
  a.workers = norm_backward_workers(a.T, a.H);
  const unsigned grid = unsigned(p.one_wave ? (a.workers + kRowWaves - 1) / kRowWaves : a.workers);
  return bf16 ? launch_backward<bf16_t>(a, p, grid, st) : launch_backward<float>(a, p, grid, st);
}

}  // namespace moe
