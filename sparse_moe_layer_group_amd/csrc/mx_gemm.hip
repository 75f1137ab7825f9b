// Products of microscaled operands by tiles, tokens by 4-bit weights, for what
// mx_stream.hip has too many tokens for.
//
//   out = residual + act(x w^T + bias), or the quantised act(x w^T) * (x w2^T)
//
// Bound by the matrix cores and the copies that feed them: a
// v_mfma_scale_f32_16x16x128_f8f6f4 of 4-bit operands takes 16 cycles, with an 8-bit
// one 32; alone they reach 6.7 and 4.4 PFLOP/s here.  Workgroup tile TM x TN, four
// waves in 2 x 2, the contraction in steps of 128 (one instruction's) through a
// ring of LDS stages filled by buffer_load ... lds copies.  A wave keeps a step's
// operands in registers and reads the next step's while it multiplies: a row
// block's are replaced as soon as its products are issued, the weights have two
// sets.  One barrier a step, after the first row blocks, when the reads of the
// stage before have long returned: behind it the next step's copies have landed
// everywhere and the stage just read is free.
//
// Stages.  Rows of 128 bytes (8 bits): 16-byte chunk c of row r at c ^ (r & 7).
// Rows of 64 (4 bits): two to a line of 128, chunk c of row r at
// (4 (r & 1) + c) ^ (r / 2 & 7).  The 16 lanes of a read's turn then have all banks
// once (counted with scales, copies and the epilogue, conflicts are 9 to 15% of the
// LDS's cycles).  Scales come four steps at a time, 16 bytes a row, and are turned
// about in LDS so that a lane reads a word with its block's of all four.
//
// Bounds.  A resource starts at the step's own first byte and ends with the
// tile's last row, so rows past the end read as zero; rows are whole steps.
// Copies of steps past the last read what follows there, or zeros, and are not
// used.
//
// Outputs are stored past the caches, which then keep the operands for the tiles to
// come (us a call without a residual, stored so and not): 8192 x 7168 x 7168 305 and
// 318, in 4 bits 220 and 251; 8192 x 2048 x 7168 113 and 123, 90 and 104; 2048 x 2048 x
// 7168 29 and 31; 17 to 1024 tokens within 0.6 either way.  With a norm behind it that
// reads the output: 8192 x 7168 x 7168 392 and 397, 4 bits 317 and 326, 2048 85 and 88,
// 17 to 1024 tokens within 0.4.  (The residual copied past them too: 132 instead of 124
// for 8192 x 2048 x 7168 with 4 bits.)
//
// Measured (tokens x in x out, us a call with a residual, calls running on): 8192 x
// 7168 x 7168, 8-bit tokens 325 (2.6 PFLOP/s), 4-bit 246 (3.4); 4096 x 7168 x 7168 158 to
// 165 and 116; 8192 x 7168 x 2048 84 and 63; 8192 x 2048 x 7168 127 and 104, of which
// the residual, 117 MB, is 20.  The first hundred or so calls after a pause take longer,
// as kernels as well: 4096 x 7168 x 7168 191, then 177, then 162.  A 256 x 256 tile's step
// takes 1.32 and 0.92 us; without its copies 1.06 and 0.69, without its LDS reads too 0.97
// and 0.62, the instructions' own time at the clock that this load leaves.  Matrix cores
// busy by counters: gate and up of 8192 tokens 59% of the time, 4096 x 7168 x 7168 51%
// (448 tiles, 1.75 turns of the chip), 8192 x 7168 x 2048 in 4 bits 30%, a single turn of
// 52 us in the loop and some 12 beside it, and what bias, residual and output take.
// float32 outputs of 8-bit tokens: 4096 x 7168 x 7168 595, 1024 170, 333 122, 50 33; of
// 4-bit ones, whose epilogue has neither image nor rows ahead, 162, 47, 23 and 14.
// Measured and not kept: copies staggered over the waves or issued early in a step
// (equal or slower), eight stages (no change), waves in two groups that split the
// contraction (no gain), 32x32x64 instructions (no faster).
#include <type_traits>

#include "dense_tiles.h"
#include "mx.h"

namespace moe {

namespace {

typedef __attribute__((address_space(3))) i32x4 lds_i32x4;
typedef __attribute__((address_space(3))) u32x4 lds_u32x4;
typedef __attribute__((address_space(3))) int lds_int;

constexpr int kThreads = 256;  // four waves, 2 x 2

template <int FORM_, int TM_, int TN_, bool DUAL_, bool EXACT_> struct MxShape {
  static constexpr int FORM = FORM_, TM = TM_, TN = TN_;
  static constexpr bool DUAL = DUAL_, EXACT = EXACT_;
  static constexpr int XB = mx_step_bytes(FORM);
  static constexpr int XS = TM * XB, WS = TN * 64;  // codes of a stage
  static constexpr int STAGE = XS + WS;
  static constexpr int XCP = XS / 4096, WCP = WS / 4096, COPIES = XCP + WCP;  // of a wave
  static constexpr int SCALES = 16 * (TM + TN);     // bytes for four steps
  // (two workgroups on a CU, but for the largest tile)
  static constexpr int FIT = ((TM * TN > 128 * 128 ? 160 : 80) * 1024 - SCALES) / STAGE;
  static constexpr int STAGES = FIT < 4 ? FIT : 4;  // (with more, scales would not have landed in time)
  static constexpr int LDS = STAGES * STAGE + SCALES;
  static_assert(STAGES >= 3 && STAGES * COPIES < 62, "vmcnt has 6 bits");
  static_assert(!DUAL || TN >= 128, "a wave has whole blocks of the product's columns");
  // a tile's rows of bfloat16 fit the stages, whole 16 of them a stage (smaller tiles
  // have another workgroup on their CU instead: 8192 x 2048 x 7168 by 128 x 128 143 us,
  // with the image 165, 45 registers out to memory)
  static constexpr bool IMAGE = !DUAL && TM * TN > 128 * 128;
  static_assert(!IMAGE || (STAGES * STAGE >= 2 * TM * TN && STAGE % (16 * 2 * TN) == 0 && XS % 1024 == 0));
  // accumulators past what 256 registers hold beside the operands: written as
  // assembly, which updates them where they lie
  static constexpr bool IN_PLACE = !EXACT;
  static constexpr bool SPLITS = TM * TN <= 128 * 128;
};

// acc += w x.  As assembly for the reason that dense_gemm.hip has: the compiler
// knows of no wait that such a product needs, so operands and scales come
// straight from LDS reads, and settle() is between it and other accesses.
template <int FORM, int BYTE> MOE_DEV void mx_multiply_add(f32x4& acc, i32x4 w, i32x8 x, int sw, int sx) {
  const i32x4 x4 = __builtin_shufflevector(x, x, 0, 1, 2, 3);
#define MOE_MX_MFMA(SEL)                                                                                         \
  if constexpr (FORM == kMxE4M3)                                                                                 \
    asm volatile("v_mfma_scale_f32_16x16x128_f8f6f4 %0, %1, %2, %0, %3, %4 " SEL " cbsz:4"                       \
                 : "+a"(acc) : "v"(w), "v"(x), "v"(sw), "v"(sx));                                                \
  else                                                                                                           \
    asm volatile("v_mfma_scale_f32_16x16x128_f8f6f4 %0, %1, %2, %0, %3, %4 " SEL " cbsz:4 blgp:4"                \
                 : "+a"(acc) : "v"(w), "v"(x4), "v"(sw), "v"(sx))
  if constexpr (BYTE == 0) { MOE_MX_MFMA("op_sel_hi:[0,0,0]"); }
  else if constexpr (BYTE == 1) { MOE_MX_MFMA("op_sel:[1,1,0] op_sel_hi:[0,0,0]"); }
  else if constexpr (BYTE == 2) { MOE_MX_MFMA("op_sel_hi:[1,1,0]"); }
  else { MOE_MX_MFMA("op_sel:[1,1,0] op_sel_hi:[1,1,0]"); }
#undef MOE_MX_MFMA
}

// A resource of what is the same in all lanes, where this compiler would put it
// into vector registers, which the copies cannot take.  left < 0: empty
MOE_DEV __amdgpu_buffer_rsrc_t scalar_rsrc(const uint8_t* p, int left) {
  const uint64_t v = reinterpret_cast<uint64_t>(p);
  uint32_t lo = __builtin_amdgcn_readfirstlane(uint32_t(v)), hi = __builtin_amdgcn_readfirstlane(uint32_t(v >> 32));
  int n = __builtin_amdgcn_readfirstlane(max(left, 0));
  // five cycles between a scalar's write by a vector instruction and its use by a
  // copy, which the compiler does not know for one
  asm volatile("s_nop 4" : "+s"(lo), "+s"(hi), "+s"(n));
  return buffer_rsrc(reinterpret_cast<const void*>(uint64_t(hi) << 32 | lo), uint32_t(n));
}

// byte s of word q to byte q of word s
MOE_DEV u32x4 transpose_bytes(u32x4 d) {
  const uint32_t a = __builtin_amdgcn_perm(d[1], d[0], 0x05010400u), b = __builtin_amdgcn_perm(d[1], d[0], 0x07030602u);
  const uint32_t c = __builtin_amdgcn_perm(d[3], d[2], 0x05010400u), e = __builtin_amdgcn_perm(d[3], d[2], 0x07030602u);
  return u32x4{__builtin_amdgcn_perm(c, a, 0x05040100u), __builtin_amdgcn_perm(c, a, 0x07060302u),
               __builtin_amdgcn_perm(e, b, 0x05040100u), __builtin_amdgcn_perm(e, b, 0x07060302u)};
}

// Columns n .. n+7 of a row of the gated product, its codes and scales: a quad of
// lanes has a block.  Padding (columns from N) is zeros.
template <int FORM> MOE_DEV void mx_gated(const MxArgs& g, int64_t m, int n, float (&v)[8], const float (&u)[8]) {
  act_values(g.epi.act, v);
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = n + i < g.N ? v[i] * u[i] : 0.f;
  const uint32_t byte = mx_quad_scale<FORM>(v);
  constexpr int W = MxForm<FORM>::WORDS;
  uint32_t o[W];
  mx_encode8<FORM>(v, byte, o);
  const int64_t piece = m * (((g.N + 127) & ~127) / 8) + n / 8;
  uint32_t* to = reinterpret_cast<uint32_t*>(g.codes) + piece * W;
  if constexpr (W == 2) *reinterpret_cast<uint2*>(to) = uint2{o[0], o[1]};
  else *to = o[0];
  if (((n / 8) & 3) == 0) g.scales[piece / 4] = uint8_t(byte);
}

// A wave's MB x NB blocks through the tile's image (its rows from `row`, its
// columns from `col` there): the residual's values, where they are there (joins),
// give way to the results in their places, and rows of these go out 16 bytes a
// lane.  m, n: of its first element in the output.
template <int TN, int MB, int NB>
MOE_DEV void image_epilogue(const MxArgs& g, lds_u8* image, f32x4 (&acc)[MB][NB], int64_t m, int n, int row, int col,
                            bool joins) {
  typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
  typedef __attribute__((address_space(3))) u32x2 lds_u32x2;
  constexpr int RB = 2 * TN, MASK = RB / 16 < 16 ? RB / 16 - 1 : 15;  // bytes of a row; of the chunks' places
  constexpr int LPR = 2 * NB, RPI = 64 / LPR;  // lanes of a wave's part of a row, rows at a time
  const int lane = threadIdx.x & 63, r16 = lane & 15, q = lane >> 4;
  float bias[NB][4];
#pragma unroll
  for (int j = 0; j < NB; ++j)
#pragma unroll
    for (int v = 0; v < 4; ++v) bias[j][v] = g.epi.bias ? load1(g.epi, g.epi.bias, n + 16 * j + 4 * q + v) : 0.f;
  lds_u8* mine = image + (row + r16) * RB + (q & 1) * 8;
  const int chunk = col / 8 + (q >> 1);
  auto place = [&](int i, int j) { return (lds_u32x2*)(mine + i * (16 * RB) + ((chunk + 2 * j) ^ (r16 & MASK)) * 16); };
  bf16_t* out = static_cast<bf16_t*>(g.epi.out) + (m + lane / LPR) * g.epi.ld_out + n + 8 * (lane % LPR);
#pragma unroll 1
  for (int i = 0; i < MB; ++i) {
    f32x4 row16[NB];
#pragma unroll
    for (int k = 0; k < MB; ++k) {
      if (k != i) continue;  // uniform: the accumulators are indexed at compile time, the rest is one loop
#pragma unroll
      for (int j = 0; j < NB; ++j) row16[j] = acc[k][j];
    }
#pragma unroll
    for (int j = 0; j < NB; j += 2) {
      float v[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) v[k] = row16[j + k / 4][k % 4] + bias[j + k / 4][k % 4];
      if (g.epi.act != kActNone) act_values(g.epi.act, v);
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        if (joins) {
          const u32x2 x = *place(i, j + h);
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            v[4 * h + 2 * k] += __uint_as_float(x[k] << 16);
            v[4 * h + 2 * k + 1] += __uint_as_float(x[k] & 0xffff0000u);
          }
        }
        *place(i, j + h) = u32x2{pack_bf16(v[4 * h], v[4 * h + 1]), pack_bf16(v[4 * h + 2], v[4 * h + 3])};
      }
    }
#pragma unroll
    for (int k = 0; k < 16 / RPI; ++k) {
      const int r = 16 * i + RPI * k + lane / LPR;
      const u32x4 x = *(lds_u32x4*)(image + (row + r) * RB + ((col / 8 + lane % LPR) ^ (r & MASK)) * 16);
      put_vector<true>(reinterpret_cast<u32x4_at2*>(out + (16 * i + RPI * k) * g.epi.ld_out), x);
    }
  }
}

}  // namespace

template <class S> __global__ __launch_bounds__(kThreads, 1) void mx_gemm_kernel(MxArgs g) {
  constexpr int TM = S::TM, TN = S::TN, XB = S::XB;
  constexpr int MB = TM / 32, NB = TN / 32;          // 16 x 16 blocks of a wave
  constexpr int NCOL = S::DUAL ? TN / 2 : TN;        // output columns of a tile
  constexpr bool WIDE = S::FORM == kMxE4M3;
  extern __shared__ __attribute__((aligned(16))) uint8_t smem[];
  lds_u8* lds = (lds_u8*)smem;

  const int mt = int((g.T + TM - 1) / TM);
  const int nt = ((S::DUAL ? (g.N + 127) & ~127 : g.N) + NCOL - 1) / NCOL;  // (dual: the padding is written too)
  int im, in;
  tile_of(blockIdx.x, mt * nt, mt, nt, im, in);
  const int64_t m0 = int64_t(im) * TM;
  const int n0 = in * NCOL;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave >> 1, wn = wave & 1;
  const int r16 = lane & 15, q = lane >> 4;
  // this workgroup's steps
  const int first = S::SPLITS ? blockIdx.y * g.steps_per_split : 0;
  const int count = S::SPLITS ? min(g.steps_per_split, g.steps - first) : g.steps;

  // ---- copy sources: offsets from the step's first byte.  Copy i of wave w
  // fills 1 KB i + w * (copies of a wave); lane l writes bytes 16 l of it.
  const uint32_t ld_x = uint32_t(g.steps) * XB, ld_w = uint32_t(g.steps) * 64u, ld_s = uint32_t(g.steps) * 4u;
  uint32_t xoff[S::XCP], woff[S::WCP];
  const int line = lane >> 3, at = (lane & 7) ^ line;  // (of 128 bytes; 8 lines a copy)
  const uint32_t xfirst = WIDE ? line * ld_x + at * 16 : (2 * line + (at >> 2)) * ld_x + (at & 3) * 16;
  const uint32_t wfirst = (2 * line + (at >> 2)) * ld_w + (at & 3) * 16;
  constexpr int XR = 1024 / XB;  // rows of a copy
#pragma unroll
  for (int i = 0; i < S::XCP; ++i) xoff[i] = (S::XCP * wave + i) * XR * ld_x + xfirst;
  // (dual: waves 0, 1 copy the first matrix's rows, 2, 3 the second's)
#pragma unroll
  for (int i = 0; i < S::WCP; ++i) woff[i] = (S::WCP * (S::DUAL ? wave & 1 : wave) + i) * 16 * ld_w + wfirst;
  // Scales, 64 rows a copy; where a tile has fewer than 256, waves copy the same ones.
  const int xsrow = (64 * wave) % TM, wsrow = (64 * wave) % TN;
  const uint32_t sxoff = (xsrow + lane) * ld_s;
  const bool second = S::DUAL && wave >= 2;         // of the weight rows that this wave copies
  const bool second_s = S::DUAL && wsrow >= TN / 2;  // (their scales)
  const uint32_t swoff = uint32_t((second_s ? wsrow - TN / 2 : wsrow) + lane) * ld_s;
  // (read as scalars: a resource made of what the compiler takes for a lane's own cannot be the copies' operand)
  const int rows_x = __builtin_amdgcn_readfirstlane(int(std::min<int64_t>(TM, g.T - m0)));
  const int rows_w = __builtin_amdgcn_readfirstlane(max(0, min(NCOL, g.N - n0)));
  const uint8_t* px = g.x + m0 * ld_x + first * XB;
  const uint8_t* psx = g.sx + m0 * ld_s + first * 4;
  const uint8_t* pw = (second ? g.w2 : g.w) + int64_t(n0) * ld_w + first * 64;
  const uint8_t* psw = (second_s ? g.sw2 : g.sw) + int64_t(n0) * ld_s + first * 4;
  // (the bytes left from there to the end of the tile's last row)
  const int all_x = rows_x * int(ld_x) - first * XB, all_w = rows_w * int(ld_w) - first * 64;
  const int all_sx = rows_x * int(ld_s) - first * 4, all_sw = rows_w * int(ld_s) - first * 4;
  int copied = 0, copied_scales = 0;  // steps, and steps of scales
  __amdgpu_buffer_rsrc_t rx = buffer_rsrc(px, max(all_x, 0)), rw = buffer_rsrc(pw, max(all_w, 0));

  // A whole tile of bfloat16 rows goes out through an image of it in LDS, over the
  // stages: rows of RB bytes, 16-byte chunk c of row r at c ^ (r & MASK).  The
  // residual's tile comes in there by the last STAGES steps' copies, which have
  // no more operands to fetch.
  constexpr int RB = 2 * TN, MASK = RB / 16 < 16 ? RB / 16 - 1 : 15, IR = 1024 / RB;  // IR: rows of a copy
  const bool whole = m0 + TM <= g.T && (S::DUAL || n0 + NCOL <= g.N);
  const bool image = S::IMAGE && whole && !g.epi.f32 && g.split == 1;
  const bf16_t* res = static_cast<const bf16_t*>(g.epi.residual);
  const uint32_t ld_res = uint32_t(g.epi.ld_residual) * 2u;
  const bool joins = image && res != nullptr && g.steps >= S::STAGES && (ld_res & 15) == 0 &&
                     (reinterpret_cast<uintptr_t>(res) & 15) == 0;
  const uint8_t* pres = reinterpret_cast<const uint8_t*>(res + m0 * g.epi.ld_residual + n0);
  const int all_res = int((TM - 1) * ld_res) + TN * 2;
  bool tail = false;
  auto take_residual = [&](int stage) __attribute__((always_inline)) {  // the rows whose place this stage is
    const int skip = stage / RB * int(ld_res);
    rx = rw = buffer_rsrc(pres + skip, max(all_res - skip, 0));
  };
  auto enter_tail = [&](int stage) __attribute__((always_inline)) {
    tail = true;
#pragma unroll
    for (int i = 0; i < S::XCP + S::WCP; ++i) {
      const int kb = i < S::XCP ? S::XCP * wave + i : S::XS / 1024 + S::WCP * wave + i - S::XCP;
      const int row = IR * kb + lane / (RB / 16);
      const uint32_t off = row * ld_res + ((lane % (RB / 16)) ^ (row & MASK)) * 16;
      if (i < S::XCP) xoff[i] = off;
      else woff[i - S::XCP] = off;
    }
    take_residual(stage);
  };
  auto advance = [&](int stage) __attribute__((always_inline)) {  // stage: the next step's
    px += XB;
    pw += 64;
    ++copied;
    if (S::IMAGE && tail) {
      take_residual(stage);
    } else {
      rx = buffer_rsrc(px, max(all_x - copied * XB, 0));
      rw = buffer_rsrc(pw, max(all_w - copied * 64, 0));
    }
  };
  // copy c of the step into the stage at `stage`
  auto copy = [&](int c, int stage) __attribute__((always_inline)) {
    if (c < S::XCP) copy_to_lds_async16(rx, xoff[c], smem + stage + (S::XCP * wave + c) * 1024);
    else copy_to_lds_async16(rw, woff[c - S::XCP], smem + stage + S::XS + (S::WCP * wave + c - S::XCP) * 1024);
  };
  // the scales of the next four steps (a row's 16 bytes begin at a multiple of 4)
  constexpr int SCALES = S::STAGES * S::STAGE;
  auto copy_scales = [&]() __attribute__((always_inline)) {
    copy_to_lds_async16(scalar_rsrc(psx + 4 * copied_scales, all_sx - 4 * copied_scales), sxoff,
                        smem + SCALES + 16 * xsrow);
    copy_to_lds_async16(scalar_rsrc(psw + 4 * copied_scales, all_sw - 4 * copied_scales), swoff,
                        smem + SCALES + 16 * (TM + wsrow));
    copied_scales += 4;
  };
  // A row's scales lie by step and block of the step; a lane needs its own block's,
  // of which the instruction picks the step's byte: each thread turns its rows
  // about, in place.
  constexpr int TURNS = (TM + TN + kThreads - 1) / kThreads;
  u32x4 turned[TURNS];
  auto scale_row = [&](int k) { return (lds_u32x4*)(lds + SCALES + 16 * (tid + k * kThreads)); };
  auto turn_read = [&]() __attribute__((always_inline)) {
#pragma unroll
    for (int k = 0; k < TURNS; ++k)
      if ((k + 1) * kThreads <= TM + TN || tid + k * kThreads < TM + TN) turned[k] = *scale_row(k);
  };
  auto turn_write = [&]() __attribute__((always_inline)) {
#pragma unroll
    for (int k = 0; k < TURNS; ++k)
      if ((k + 1) * kThreads <= TM + TN || tid + k * kThreads < TM + TN) *scale_row(k) = transpose_bytes(turned[k]);
  };

  // ---- fragments
  f32x4 acc[MB][NB];
  i32x8 xf[MB];
  i32x4 wf[2][NB];
  int sx[MB], sw[NB], next_sw[NB];
  // first staged weight row of the wave's block j: a dual wave takes the same
  // columns of both matrices
  auto wrow = [&](int j) {
    return S::DUAL ? (j / (NB / 2)) * (TN / 2) + wn * (TN / 4) + 16 * (j % (NB / 2)) : wn * (TN / 2) + 16 * j;
  };
  const int half = (4 * (r16 & 1) + q) ^ (r16 >> 1);  // chunk of a row of 64 bytes in its line
  const int xrow = wm * (TM / 2) + r16;
  const int xlo = WIDE ? xrow * 128 + (q ^ (r16 & 7)) * 16 : (xrow >> 1) * 128 + half * 16;
  const int xhi = xrow * 128 + ((q ^ 4) ^ (r16 & 7)) * 16;
  const int wat = S::XS + ((wrow(0) + r16) >> 1) * 128 + half * 16;
  const int sxat = SCALES + 16 * xrow + 4 * q, swat = SCALES + 16 * (TM + wrow(0) + r16) + 4 * q;
  // (scales: the step is the first of four)
  auto read_x = [&](int i, int stage, bool scales) __attribute__((always_inline)) {
    const i32x4 lo = *(const lds_i32x4*)(lds + stage + xlo + i * 16 * XB);
    i32x4 hi = lo;
    if (WIDE) hi = *(const lds_i32x4*)(lds + stage + xhi + i * 16 * XB);
    xf[i] = __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
    if (scales) sx[i] = *(const lds_int*)(lds + sxat + i * 256);
  };
  auto read_w = [&](int set, int j, int stage, bool scales) __attribute__((always_inline)) {
    const int row = wrow(j) - wrow(0);
    wf[set][j] = *(const lds_i32x4*)(lds + stage + wat + row * 64);
    if (scales) next_sw[j] = *(const lds_int*)(lds + swat + row * 16);
  };
  auto multiply = [&](auto byte, int set, int i, int j) __attribute__((always_inline)) {
    constexpr int BYTE = decltype(byte)::value;
    if constexpr (S::IN_PLACE) {
      mx_multiply_add<S::FORM, BYTE>(acc[i][j], wf[set][j], xf[i], sw[j], sx[i]);
    } else {
      const i32x4 lo = __builtin_shufflevector(xf[i], xf[i], 0, 1, 2, 3);
      const i32x4 hi = __builtin_shufflevector(xf[i], xf[i], 4, 5, 6, 7);
      acc[i][j] = mx_multiply<S::FORM, S::EXACT, BYTE>(wf[set][j], sw[j], lo, hi, sx[i], acc[i][j]);
    }
  };

  // ---- the loop
  copy_scales();
#pragma unroll
  for (int st = 0; st < S::STAGES; ++st) {
#pragma unroll
    for (int c = 0; c < S::COPIES; ++c) copy(c, st * S::STAGE);
    advance(0);
  }
#pragma unroll
  for (int i = 0; i < MB; ++i)
#pragma unroll
    for (int j = 0; j < NB; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
  if constexpr (S::IN_PLACE) settle(acc);
  __builtin_amdgcn_s_waitcnt(wait_copies((S::STAGES - 1) * S::COPIES));
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
  turn_read();
  turn_write();
  __builtin_amdgcn_s_waitcnt(wait_copies((S::STAGES - 1) * S::COPIES) & ~0xf00);
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
#pragma unroll
  for (int j = 0; j < NB; ++j) {
    read_w(0, j, 0, true);
    sw[j] = next_sw[j];
  }
#pragma unroll
  for (int i = 0; i < MB; ++i) read_x(i, 0, true);

  constexpr int SYNC = MB >= 4 ? 2 : 1;  // row blocks before the barrier
  constexpr int G = (MB - SYNC) * NB;    // products after it
  int now = 0, next = S::STAGE;          // stages of this step and the next
  // Step PH of four.  The first issues the copies of the next four's scales before
  // its others; by the third they have landed and are turned about there, and in
  // the fourth they are read.
  auto step = [&](auto ph_) __attribute__((always_inline)) {
    constexpr int PH = decltype(ph_)::value, set = PH & 1;
    // copies since those of the next step's codes; by the third step, and since the scales'
    constexpr int LATER = (S::STAGES - 2) * S::COPIES + (PH == 1 ? 2 : 0);
#pragma unroll
    for (int i = 0; i < MB; ++i) {
      if (i == SYNC) {
        // this wave's copies of the next step have landed (those of later steps
        // are in flight) and its reads of this step's stage are done; behind the
        // barrier everyone's
        __builtin_amdgcn_s_waitcnt(wait_copies(LATER) & ~0xf00);
        __builtin_amdgcn_s_barrier();
        asm volatile("" ::: "memory");
      }
#pragma unroll
      for (int jj = 0; jj < NB; ++jj) {
        multiply(ph_, set, i, i & 1 ? NB - 1 - jj : jj);  // one operand stays at every turn
        if (i >= SYNC) {
          const int t = (i - SYNC) * NB + jj;
          if (PH == 0 && t == 0) copy_scales();
#pragma unroll
          for (int r = 0; r < NB; ++r)
            if (t == r * G * 2 / (3 * NB)) read_w(set ^ 1, r, next, PH == 3);
          if (jj == 0) read_x(i - SYNC, next, PH == 3);
#pragma unroll
          for (int r = MB - SYNC; r < MB - 1; ++r)
            if (i == MB - 1 && jj == NB / 2) read_x(r, next, PH == 3);
#pragma unroll
          for (int c = 0; c < S::COPIES; ++c)
            if (t == (c * G + G / 2) / S::COPIES) copy(c, now);
          if (PH == 2 && t == 0) turn_read();
          if (PH == 2 && t == G / 2) turn_write();
        }
        __builtin_amdgcn_sched_barrier(0);
      }
    }
    read_x(MB - 1, next, PH == 3);
    advance(next);
    if (PH == 3) {
#pragma unroll
      for (int j = 0; j < NB; ++j) sw[j] = next_sw[j];
    }
    now = next;
    next = next == (S::STAGES - 1) * S::STAGE ? 0 : next + S::STAGE;
  };
  int left = count;
  auto begin = [&]() __attribute__((always_inline)) {
    if (S::IMAGE && joins && left == S::STAGES) enter_tail(now);
  };
  for (;;) {
    begin();
    step(std::integral_constant<int, 0>{});
    if (--left == 0) break;
    begin();
    step(std::integral_constant<int, 1>{});
    if (--left == 0) break;
    begin();
    step(std::integral_constant<int, 2>{});
    if (--left == 0) break;
    begin();
    step(std::integral_constant<int, 3>{});
    if (--left == 0) break;
  }
  if constexpr (S::IN_PLACE) settle(acc);
  __builtin_amdgcn_s_waitcnt(kWaitAll);  // no copy left in flight
  __syncthreads();

  // ---- epilogue.  The weights are the instruction's first operand, so
  // accumulator v of lane l is row l % 16, column 4 (l / 16) + v.
  if constexpr (S::IMAGE) {
    if (image && (joins || res == nullptr)) {
      image_epilogue<TN, MB, NB>(g, lds, acc, m0 + wm * (TM / 2), n0 + wn * (TN / 2), wm * (TM / 2), wn * (TN / 2), joins);
      return;
    }
  }
  // Each wave passes 32 rows of its columns at a time through LDS (float32), so that a
  // lane has 8 consecutive columns of a row.
  constexpr int WC = 16 * NB, OC = S::DUAL ? WC / 2 : WC, PITCH = WC * 4 + 16;
  static_assert(4 * 32 * PITCH <= S::LDS, "the staging rows fit the stages");
  constexpr int LPR = OC / 8, RPI = 64 / LPR;  // lanes of a row, rows at a time
  lds_u8* rows32 = lds + wave * 32 * PITCH;
  const int c = 8 * (lane % LPR), n = n0 + wn * OC + c;
  constexpr int MODE = S::DUAL ? kEpiGated : kEpiOut;
  float bias[1][8], total[8];  // (total: another mode's)
  load_bias<MODE, false>(g.epi, n, bias);
  // R rows of this lane from row r of the staged 32, which are rows mrow ...
  auto finish = [&](int64_t mrow, int r, auto inside, auto rows) __attribute__((always_inline)) {
    constexpr int R = decltype(rows)::value;
    float v[R][8], u[R][8];
#pragma unroll
    for (int k = 0; k < R; ++k)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const lds_u8* from = rows32 + (r + k * RPI) * PITCH + 4 * c + 16 * h;
        const f32x4 p = *(const lds_f32x4*)from;
        f32x4 p2 = {0.f, 0.f, 0.f, 0.f};
        if (S::DUAL) p2 = *(const lds_f32x4*)(from + 4 * OC);
#pragma unroll
        for (int i = 0; i < 4; ++i) { v[k][4 * h + i] = p[i]; u[k][4 * h + i] = p2[i]; }
      }
    if (S::SPLITS && g.split > 1) {
#pragma unroll
      for (int k = 0; k < R; ++k) {
        float* to = g.part + (int64_t(blockIdx.y) * (S::DUAL ? 2 : 1) * g.T + mrow + r + k * RPI) * g.ld_part + n;
        store8<true>(to, 0, 8, v[k]);
        if (S::DUAL) store8<true>(to + g.T * g.ld_part, 0, 8, u[k]);
      }
      return;
    }
    if constexpr (S::DUAL) {
#pragma unroll
      for (int k = 0; k < R; ++k) mx_gated<S::FORM>(g, mrow + r + k * RPI, n, v[k], u[k]);
    } else {
      dense_epilogue<kEpiOut, decltype(inside)::value, R, true>(g.epi, mrow + r, RPI, n, v, u, bias, total);
    }
  };
  // rows at a time where all are inside
  constexpr int AHEAD = S::IMAGE ? 1 : 32 / RPI < 4 ? 32 / RPI : 4;
  const int64_t row0 = m0 + wm * (TM / 2);
#pragma unroll 1
  for (int blk = 0; blk < MB / 2; ++blk) {
    const int64_t mrow = row0 + 32 * blk;
    if (mrow >= g.T) break;  // uniform
#pragma unroll
    for (int i = 0; i < MB; ++i) {
      if (i / 2 != blk) continue;  // uniform: the accumulators are indexed at compile time, the rest is one loop
#pragma unroll
      for (int j = 0; j < NB; ++j)
        *(lds_f32x4*)(rows32 + (16 * (i & 1) + r16) * PITCH + 4 * (16 * j + 4 * q)) = acc[i][j];
    }
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    if (mrow + 32 <= g.T && (S::DUAL || n0 + wn * OC + OC <= g.N)) {  // (this wave's, in a tile that is not whole too)
#pragma unroll 1
      for (int r = lane / LPR; r < 32; r += RPI * AHEAD)
        finish(mrow, r, std::true_type{}, std::integral_constant<int, AHEAD>{});
    } else if (S::DUAL || n < g.N) {
#pragma unroll 1
      for (int r = lane / LPR; r < 32; r += RPI)
        if (mrow + r < g.T) finish(mrow, r, std::false_type{}, std::integral_constant<int, 1>{});
    }
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
  }
}

// Sums of a split contraction, in order, and the epilogue on them: eight columns
// of a row a lane.
constexpr int kJoinThreads = 64;  // (as many workgroups as there are for few rows)
template <int FORM, bool DUAL> __global__ __launch_bounds__(kJoinThreads) void mx_join_kernel(MxArgs g) {
  const uint32_t pieces = uint32_t(g.ld_part) / 8;  // of a row: whole quads of lanes
  const uint32_t id = blockIdx.x * kJoinThreads + threadIdx.x, row = id / pieces;
  const int64_t m = row;
  const int n = int(id - row * pieces) * 8;
  if (m >= g.T) return;
  float v[1][8], u[1][8];
#pragma unroll
  for (int i = 0; i < 8; ++i) v[0][i] = u[0][i] = 0.f;
  const int64_t part = g.T * g.ld_part;
#pragma unroll 8
  for (int s = 0; s < g.split; ++s) {
    const float* p = g.part + s * (DUAL ? 2 : 1) * part + m * g.ld_part + n;
    float x[8], y[8];
    load8<true>(p, 0, 8, x);
    if (DUAL) load8<true>(p + part, 0, 8, y);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      v[0][i] += x[i];
      if (DUAL) u[0][i] += y[i];
    }
  }
  if constexpr (DUAL) {
    mx_gated<FORM>(g, m, n, v[0], u[0]);
  } else if (n < g.N) {
    float b[1][8], total[8] = {};
    load_bias<kEpiOut, false>(g.epi, n, b);
    dense_epilogue<kEpiOut, false, 1>(g.epi, m, 0, n, v, u, b, total);
  }
}

namespace {

int64_t padded_columns(const MxArgs& g) { return (int64_t(g.N) + 127) / 128 * 128; }
int64_t tiles_of(const MxArgs& g, int tm, int tn) {
  const int64_t columns = g.w2 ? 2 * padded_columns(g) : g.N;
  return (g.T + tm - 1) / tm * ((columns + tn - 1) / tn);
}

template <class S> hipError_t launch(const MxArgs& g, hipStream_t st) {
  hipLaunchKernelGGL(mx_gemm_kernel<S>, dim3(unsigned(tiles_of(g, S::TM, S::TN)), unsigned(g.split)), dim3(kThreads),
                     S::LDS, st, g);
  return hipGetLastError();
}
template <int FORM, bool EXACT, int TM, int TN> hipError_t launch_tile(const MxArgs& g, hipStream_t st) {
  if constexpr (TN < 128) {
    return launch<MxShape<FORM, TM, TN, false, EXACT>>(g, st);
  } else {
    return g.w2 ? launch<MxShape<FORM, TM, TN, true, EXACT>>(g, st) : launch<MxShape<FORM, TM, TN, false, EXACT>>(g, st);
  }
}

// A product's tile and split of the contraction, by their time in us: turns of the
// chip, each of so many steps and what a tile takes beside them; a second launch
// that joins the parts, and these through memory.  Calls measured with every tile
// forced (64 x 64, 64 x 128, 128 x 128, 256 x 256, each with the best split), 8-bit
// tokens: 50 x 7168 x 2048 10.7, 10.7, 11.6, 70.4 (not split 14.3); 333 x 7168 x 7168
// 32.9, 30.7, 28.0, 76.0; 1024 x 7168 x 2048 25.6, 21.2, 27.5, 75.4; 2048 x 7168 x 7168
// 163, 123, 104, 81.1; 4096 x 7168 x 2048 93.8, 72.4, 57.7, 76.0; 8192 x 2048 x 7168 210,
// 168, 145, 136; 8192 x 1024 x 7168 128 x 128 80.7, 256 x 256 89.9.  Of 15 sizes and both
// forms the rule took the fastest or one within 3% of it, but for 50 x 7168 x 7168 in
// 4 bits (14.2 by 64 x 64, 13.3 by 64 x 128).
// `exact` products are planned by the same figures, although a step of theirs is three
// instructions and the masks: what is taken is right for many tokens (64 x 64, 64 x 128,
// 128 x 128: 1024 x 7168 x 7168 234, 179, 170; 4096 906, 627, 594; 8192 x 2048 x 7168 560,
// 401, 384; the last is taken) and not for few (50 x 7168 x 7168 33 taken, 25 by 64 x 128;
// 333 122 taken, 91 by 64 x 128; 333 x 7168 x 2048 55 taken, 40 by 64 x 128).
struct TileCost {
  int tm, tn;  // token rows, weight rows
  float step, rest;
};
constexpr int kTiles = 4;
constexpr TileCost kCosts[2][kTiles] = {  // by form
    {{64, 64, 0.197f, 0.3f}, {64, 128, 0.292f, 0.6f}, {128, 128, 0.455f, 2.2f}, {256, 256, 1.32f, 12.f}},
    {{64, 64, 0.158f, 0.3f}, {64, 128, 0.25f, 0.6f}, {128, 128, 0.375f, 2.f}, {256, 256, 0.92f, 12.f}}};
constexpr int kMostSplit = 16, kFewest = 3;  // parts, steps of one
constexpr float kJoin = 4.f, kPartBytes = 3e6f;  // us, bytes a us
constexpr int kUnits = 256;
struct Plan {
  int tile, split, per;
};
Plan plan_of(const MxArgs& g, int form) {
  Plan best{-1, 1, g.steps};
  float least = 0.f;
  for (int i = 0; i < kTiles; ++i) {
    const TileCost& c = kCosts[form][i];
    if (g.w2 && c.tn < 128) continue;
    if (g.exact && form == kMxE4M3 && c.tm > 128) continue;
    const int64_t tiles = tiles_of(g, c.tm, c.tn);
    for (int split = 1; split <= kMostSplit; ++split) {
      const int per = (g.steps + split - 1) / split;
      if (split > 1 && (c.tm > 128 || tiles * split > kUnits || per < kFewest)) break;
      if ((g.steps + per - 1) / per != split) continue;  // the same as a smaller one's
      float time = float((tiles * split + kUnits - 1) / kUnits) * (float(per) * c.step + c.rest);
      if (split > 1) time += kJoin + float(split) * float(tiles) * float(c.tm * c.tn * 4) / kPartBytes;
      if (best.tile < 0 || time < least) {
        least = time;
        best = Plan{i, split, per};
      }
    }
  }
  return best;
}

template <int FORM, bool EXACT> hipError_t launch_form(const MxArgs& args, float* part, hipStream_t st) {
  MxArgs g = args;
  const Plan p = plan_of(g, FORM);
  g.split = p.split;
  g.steps_per_split = p.per;
  g.part = part;
  g.ld_part = padded_columns(g);
  const bool dual = g.w2 != nullptr;
  if (p.split > 1 && size_t(p.split) * (dual ? 2 : 1) * size_t(g.T) * size_t(g.ld_part) * sizeof(float) >
                         mx_part_bytes(g.T, g.N, dual))
    return hipErrorInvalidValue;  // (the plan keeps within it)
  hipError_t err;
  switch (p.tile) {
    case 0: err = launch_tile<FORM, EXACT, 64, 64>(g, st); break;
    case 1: err = launch_tile<FORM, EXACT, 64, 128>(g, st); break;
    case 2: err = launch_tile<FORM, EXACT, 128, 128>(g, st); break;
    default:
      if constexpr (EXACT) err = hipErrorInvalidValue;
      else err = launch_tile<FORM, false, 256, 256>(g, st);
  }
  if (err != hipSuccess || g.split == 1) return err;
  const unsigned grid = unsigned((g.T * (g.ld_part / 8) + kJoinThreads - 1) / kJoinThreads);  // (at most 256 tiles' rows)
  if (g.w2) hipLaunchKernelGGL((mx_join_kernel<FORM, true>), dim3(grid), dim3(kJoinThreads), 0, st, g);
  else hipLaunchKernelGGL((mx_join_kernel<FORM, false>), dim3(grid), dim3(kJoinThreads), 0, st, g);
  return hipGetLastError();
}

}  // namespace

// Parts are of at most 256 tiles of the largest that is split, and at most
// kMostSplit of the rows (up to whole tiles): grows with T.
size_t mx_part_bytes(int64_t T, int N, bool dual) {
  const size_t most = size_t(kUnits) * 128 * 128 * sizeof(float);
  const size_t rows = (size_t(T) + 127) / 128 * 128, columns = (size_t(N) + 127) / 128 * 128 * (dual ? 2 : 1);
  return std::min(most, size_t(kMostSplit) * rows * columns * sizeof(float));
}

hipError_t launch_mx_gemm(const MxArgs& g, int form, float* part, hipStream_t st) {
  if (g.T < 1 || g.N < 1 || g.steps < 1) return hipErrorInvalidValue;
  if (form == kMxE2M1) return launch_form<kMxE2M1, false>(g, part, st);
  return g.exact ? launch_form<kMxE4M3, true>(g, part, st) : launch_form<kMxE4M3, false>(g, part, st);
}

}  // namespace moe
