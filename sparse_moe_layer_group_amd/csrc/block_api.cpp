// C ABI of the operators around the expert layer (norms with the residual
// stream, projections, the dense gated feed-forward block): argument checks,
// workspace layout and launch order.  The work is in norm_kernels.hip and
// dense_gemm.hip.
#include <hip/hip_runtime.h>

#include <atomic>
#include <cmath>
#include <cstring>

#include "../../include/moe.h"
#include "block.h"

namespace {

using moe::bf16_t;

constexpr int64_t kMaxRows = int64_t(1) << 24, kMaxLd = int64_t(1) << 22;
constexpr int32_t kMaxDim = 131072;

#define MOE_TRY(expr)                             \
  do {                                            \
    if ((expr) != hipSuccess) return MOE_ERR_HIP; \
  } while (0)

// the current device is a gfx950 GPU (cached per device)
int check_device() {
  static std::atomic<int> state[64];
  int dev = 0;
  if (hipGetDevice(&dev) != hipSuccess) return MOE_ERR_HIP;
  if (dev < 0 || dev >= 64) return MOE_ERR_DEVICE;
  int st = state[dev].load(std::memory_order_relaxed);
  if (st == 0) {
    hipDeviceProp_t prop;
    if (hipGetDeviceProperties(&prop, dev) != hipSuccess) return MOE_ERR_HIP;
    st = std::strncmp(prop.gcnArchName, "gfx950", 6) == 0 ? 1 : -1;
    state[dev].store(st, std::memory_order_relaxed);
  }
  return st == 1 ? MOE_OK : MOE_ERR_DEVICE;
}

int check_dtype(int32_t dt) { return dt == MOE_F32 || dt == MOE_BF16 ? MOE_OK : MOE_ERR_DTYPE; }
bool bad_dim(int32_t d) { return d < 1 || d > kMaxDim; }
bool bad_rows(int64_t T) { return T < 0 || T > kMaxRows; }
bool bad_ld(const void* p, int64_t ld, int64_t cols) { return p != nullptr && (ld < cols || ld >= kMaxLd); }
bool bad_ws(const void* ws, size_t have, size_t need) {
  return need > 0 && (ws == nullptr || have < need || (reinterpret_cast<uintptr_t>(ws) & 15) != 0);
}

// consecutive pieces of a workspace, 256 bytes apart
struct Carver {
  char* base;  // NULL: only the total is wanted
  size_t used = 0;
  template <typename P> P* take(size_t bytes) {
    char* p = base == nullptr ? nullptr : base + used;
    used += (bytes + 255) & ~size_t(255);
    return reinterpret_cast<P*>(p);
  }
};

// ---------------------------------------------------------------- norm

int validate(const moe_norm_cfg* c, int64_t T) {
  if (c == nullptr) return MOE_ERR_NULL;
  if (check_dtype(c->dtype) != MOE_OK) return MOE_ERR_DTYPE;
  if (c->hidden < 1 || c->hidden > moe::kNormMaxHidden) return MOE_ERR_SHAPE;
  if (c->kind != MOE_NORM_RMS && c->kind != MOE_NORM_LAYER) return MOE_ERR_SHAPE;
  if (!(c->eps >= 0.f) || !std::isfinite(c->eps) || !std::isfinite(c->res_scale)) return MOE_ERR_SHAPE;
  if (bad_rows(T) || c->gate_rows < 0 || (c->gate_rows > 0 && T % c->gate_rows != 0)) return MOE_ERR_SHAPE;
  return MOE_OK;
}

int check_params(const moe_norm_cfg& c, const moe_norm_params* p, bool branch, bool pre) {
  if (p == nullptr) return MOE_ERR_NULL;
  if (c.kind == MOE_NORM_RMS && (p->b_post != nullptr || p->b_pre != nullptr)) return MOE_ERR_SHAPE;
  if (c.gate_rows == 0 && p->gate != nullptr) return MOE_ERR_SHAPE;
  if (c.gate_rows > 0 && p->gate == nullptr) return MOE_ERR_NULL;
  if (p->b_post != nullptr && p->w_post == nullptr) return MOE_ERR_NULL;
  if (!branch && (p->w_post != nullptr || p->gate != nullptr)) return MOE_ERR_NULL;
  if (pre && p->w_pre == nullptr) return MOE_ERR_NULL;
  return MOE_OK;
}

moe::NormArgs norm_args(const moe_norm_cfg& c, int64_t T, const void* residual, int64_t ld_residual,
                        const void* branch, int64_t ld_branch, const moe_norm_params& p) {
  moe::NormArgs a{};
  a.residual = residual;
  a.branch = branch;
  a.ld_residual = ld_residual;
  a.ld_branch = ld_branch;
  a.w_post = p.w_post;
  a.b_post = p.b_post;
  a.w_pre = p.w_pre;
  a.b_pre = p.b_pre;
  a.gate = p.gate;
  a.T = T;
  a.H = c.hidden;
  a.gate_rows = c.gate_rows;
  a.layer = c.kind == MOE_NORM_LAYER;
  a.eps = c.eps;
  a.scale = c.res_scale;
  return a;
}

size_t norm_carve(const moe_norm_cfg& c, int64_t T, void* ws, moe::NormArgs& a) {
  Carver w{static_cast<char*>(ws)};
  const size_t row = size_t(c.hidden) * sizeof(float);
  const size_t n = size_t(moe::norm_backward_workers(T, c.hidden));
  a.part = w.take<float>(4 * n * row);
  a.gpart = w.take<float>(c.gate_rows > 0 ? 2 * n * row : 0);
  return w.used;
}

// ---------------------------------------------------------------- operands of the products

// A matrix as the products read it: one bfloat16 plane, or three for float32.
struct Mat {
  const bf16_t* p[3];
  int64_t ld;
};

int64_t padded(int64_t cols) { return (cols + 63) & ~int64_t(63); }
size_t planes_bytes(bool f32, int64_t rows, int64_t cols) {
  return size_t(f32 ? 3 : 1) * size_t(rows) * size_t(padded(cols)) * sizeof(bf16_t);
}
Mat planes_at(bool f32, bf16_t* p, int64_t rows, int64_t cols) {
  const int64_t ld = padded(cols);
  return Mat{{p, f32 ? p + rows * ld : p, f32 ? p + 2 * rows * ld : p}, ld};
}

// A user's matrix: as it is where the products can read it, else laid out
// anew at `room` (float32: split into planes).  The room is part of the
// workspace of every call that goes to the tiles, as its size goes by the
// configuration alone.
struct Source {
  const void* p;
  int64_t ld, rows;
  int cols;
  bf16_t* room;
};
Source source(Carver& w, bool f32, const void* p, int64_t ld, int64_t rows, int cols) {
  return Source{p, ld, rows, cols, w.take<bf16_t>(planes_bytes(f32, rows, cols))};
}
bool direct(const Source& s) {
  return s.cols % 8 == 0 && s.ld % 8 == 0 && (reinterpret_cast<uintptr_t>(s.p) & 15) == 0;
}
// The operands of a call; what has to be laid out anew is, in one launch.
struct Operands {
  bool f32;
  moe::PackJobs jobs;
  int count = 0;
  explicit Operands(bool f) : f32(f) {}
  Mat add(const Source& s, bool as_is) {
    if (!f32 && as_is) {
      const bf16_t* p = static_cast<const bf16_t*>(s.p);
      return Mat{{p, p, p}, s.ld};
    }
    const Mat m = planes_at(f32, s.room, s.rows, s.cols);
    jobs.j[count++] = moe::PackJob{s.p, s.ld, s.rows, s.cols, s.room, m.ld};
    return m;
  }
  Mat add(const Source& s) { return add(s, direct(s)); }
  hipError_t lay_out(hipStream_t st) const { return moe::launch_dense_pack(jobs, count, f32, st); }
};

// Segments of A B over the planes, smallest terms first.  Of float32's nine
// pairs, mid lo and lo mid are up to 2^-25 of the product each, lo lo 2^-34: left
// out.
constexpr int kPairs = 6;
constexpr int kPairA[kPairs] = {2, 0, 1, 1, 0, 0}, kPairB[kPairs] = {0, 2, 1, 0, 1, 0};

// appends A B (and A B2) to the segments of a product
void add_segments(moe::DenseArgs& g, bool f32, const Mat& A, const Mat& B, const Mat* B2 = nullptr) {
  g.lda = A.ld;
  g.ldb = B.ld;
  g.dual = B2 != nullptr;
  for (int i = 0; i < (f32 ? kPairs : 1); ++i) {
    const int s = g.segments++;
    const int a = f32 ? kPairA[i] : 0, b = f32 ? kPairB[i] : 0;
    g.a[s] = A.p[a];
    g.b[s] = B.p[b];
    g.b2[s] = B2 != nullptr ? B2->p[b] : nullptr;
  }
}
moe::DenseArgs product(int64_t M, int N, int64_t K, int mode, bool f32) {
  moe::DenseArgs g{};
  g.M = M;
  g.N = N;
  g.K = K;
  g.epi.mode = mode;
  g.epi.f32 = f32;
  g.epi.M = M;
  g.epi.N = N;
  return g;
}
// staged operands of a later product as an epilogue's outputs
void stage_to(moe::DenseEpi& e, const Mat& m, int64_t rows) {
  e.ld_p = m.ld;
  e.plane = rows * m.ld;
}
// Which batches a workspace is laid out for.  A call asks for its own; a query
// for its own and every smaller one, so that a workspace made once serves them
// all: the sums of split contractions, alone in this, take more room for some
// smaller batches, which have fewer tiles and more splits.
enum Batches { kThis, kUpTo };
// room for split sums of a product with T rows, and of one that contracts over T
size_t rows_part(Batches b, int64_t T, int N, int64_t K, bool f32, int pairs = 1, int dual = 0) {
  const int segments = pairs * (f32 ? kPairs : 1);
  return b == kThis ? moe::dense_part_bytes(T, N, K, segments, dual, 1, true)
                    : moe::dense_part_most(T, N, K, segments, dual, 1);
}
size_t deep_part(Batches b, int64_t M, int N, int64_t T, bool f32, int count = 1) {
  const int segments = f32 ? kPairs : 1;
  return b == kThis ? moe::dense_part_bytes(M, N, T, segments, 0, count, false)
                    : moe::dense_part_most_deep(M, N, T, segments, count);
}
hipError_t launch(const moe::DenseArgs& g, int layout, float* part, hipStream_t st) {
  moe::DenseGroup group{};
  group.g[0] = g;
  return moe::launch_dense(group, 1, layout, part, st);
}

// Whether a forward product goes to the weight-streaming kernel.  bfloat16: up
// to 16 tokens, one MFMA's (a block of hidden 7168 and inter 2048, weights from
// memory: one token 24.9 us against 26.7 by tiles, 8 26.5 against 26.8, 16 28.6
// against 27.0, 17 31.1 against 27.9, 32 39 against 29; weights of odd rows or
// unaligned ones it takes as they are, where the tiles need a copy).  float32:
// to 64, as the tiles need the weights laid out as three planes first (one token
// 46 us against 157, 64 tokens 129 against 178).
bool streams(int64_t T, bool f32) { return T <= (f32 ? moe::kStreamTokens : 16); }

// ---------------------------------------------------------------- linear

int validate(const moe_linear_cfg* c, int64_t T) {
  if (c == nullptr) return MOE_ERR_NULL;
  if (check_dtype(c->dtype) != MOE_OK) return MOE_ERR_DTYPE;
  if (bad_dim(c->in_dim) || bad_dim(c->out_dim) || bad_rows(T)) return MOE_ERR_SHAPE;
  if (c->act < MOE_ACT_NONE || c->act > MOE_ACT_GELU) return MOE_ERR_SHAPE;
  return MOE_OK;
}

struct LinearWork {
  Source x, w, dy;
  bf16_t* dz;
  float *part, *sums;
  size_t bytes;
};
LinearWork linear_carve(const moe_linear_cfg& c, Batches b, int64_t T, bool back, void* ws, const void* x,
                        int64_t ld_x, const void* w, const void* dy, int64_t ld_dy) {
  const bool f32 = c.dtype == MOE_F32;
  const int K = c.in_dim, N = c.out_dim;
  Carver v{static_cast<char*>(ws)};
  LinearWork L{};
  if (!back && streams(T, f32)) {  // nothing but a size that is not 0, which a query has for what is invalid
    v.take<char>(1);
    L.bytes = v.used;
    return L;
  }
  L.x = source(v, f32, x, ld_x, T, K);
  L.w = source(v, f32, w, K, N, K);
  size_t part = rows_part(b, T, N, K, f32);
  if (back) {
    if (c.act == MOE_ACT_NONE) L.dy = source(v, f32, dy, ld_dy, T, N);
    else L.dz = v.take<bf16_t>(planes_bytes(f32, T, N));
    part = std::max(part, rows_part(b, T, K, N, f32));
    part = std::max(part, deep_part(b, N, K, T, f32));
    L.sums = v.take<float>(moe::dense_sums_bytes(T, N));
  }
  L.part = v.take<float>(part);
  L.bytes = v.used;
  return L;
}

// ---------------------------------------------------------------- ffn

int validate(const moe_ffn_cfg* c, int64_t T) {
  if (c == nullptr) return MOE_ERR_NULL;
  if (check_dtype(c->dtype) != MOE_OK) return MOE_ERR_DTYPE;
  if (bad_dim(c->hidden) || bad_dim(c->inter) || bad_rows(T)) return MOE_ERR_SHAPE;
  if (c->act != MOE_ACT_RELU && c->act != MOE_ACT_SILU && c->act != MOE_ACT_GELU) return MOE_ERR_SHAPE;
  return MOE_OK;
}

struct FfnWork {
  Source x, wg, wu, wd, dy;
  bf16_t *mid, *dg, *du;  // staged operands [T][inter] (few tokens: mid of the call's type)
  float *g, *u;           // the projections, float32 (backward)
  float* part;
  size_t bytes;
};
FfnWork ffn_carve(const moe_ffn_cfg& c, Batches b, int64_t T, bool back, void* ws, const void* x, int64_t ld_x,
                  const void* wg, const void* wu, const void* wd, const void* dy, int64_t ld_dy) {
  const bool f32 = c.dtype == MOE_F32;
  const int H = c.hidden, I = c.inter;
  Carver v{static_cast<char*>(ws)};
  FfnWork F{};
  if (!back && streams(T, f32)) {  // packed rows of the type
    F.mid = v.take<bf16_t>(size_t(T) * size_t(I) * (f32 ? sizeof(float) : sizeof(bf16_t)));
    F.bytes = v.used;
    return F;
  }
  F.x = source(v, f32, x, ld_x, T, H);
  F.wg = source(v, f32, wg, H, I, H);
  F.wu = source(v, f32, wu, H, I, H);
  F.wd = source(v, f32, wd, I, H, I);
  F.mid = v.take<bf16_t>(planes_bytes(f32, T, I));
  size_t part = rows_part(b, T, I, H, f32, 1, 1);
  if (back) {
    F.dy = source(v, f32, dy, ld_dy, T, H);
    F.dg = v.take<bf16_t>(planes_bytes(f32, T, I));
    F.du = v.take<bf16_t>(planes_bytes(f32, T, I));
    F.g = v.take<float>(size_t(T) * size_t(padded(I)) * sizeof(float));
    F.u = v.take<float>(size_t(T) * size_t(padded(I)) * sizeof(float));
    part = std::max(part, rows_part(b, T, I, H, f32));
    part = std::max(part, rows_part(b, T, H, I, f32, 2));
    part = std::max(part, deep_part(b, I, H, T, f32, 3));
    part = std::max(part, deep_part(b, H, I, T, f32, 3));
  } else {
    part = std::max(part, rows_part(b, T, H, I, f32));
  }
  F.part = v.take<float>(part);
  F.bytes = v.used;
  return F;
}

}  // namespace

extern "C" {

// ---------------------------------------------------------------- norm

int moe_norm_forward(const moe_norm_cfg* cfg, int64_t T, const void* residual, int64_t ld_residual,
                     const void* branch, int64_t ld_branch, const moe_norm_params* params, void* u, int64_t ld_u,
                     void* h, int64_t ld_h, void* stream) {
  int rc = validate(cfg, T);
  if (rc != MOE_OK || T == 0) return rc;
  if (residual == nullptr || (u == nullptr && h == nullptr)) return MOE_ERR_NULL;
  if ((rc = check_params(*cfg, params, branch != nullptr, h != nullptr)) != MOE_OK) return rc;
  const int64_t H = cfg->hidden;
  if (bad_ld(residual, ld_residual, H) || bad_ld(branch, ld_branch, H) || bad_ld(u, ld_u, H) || bad_ld(h, ld_h, H))
    return MOE_ERR_SHAPE;
  if ((rc = check_device()) != MOE_OK) return rc;
  moe::NormArgs a = norm_args(*cfg, T, residual, ld_residual, branch, ld_branch, *params);
  a.u = u;
  a.ld_u = ld_u;
  a.h = h;
  a.ld_h = ld_h;
  MOE_TRY(moe::launch_norm_forward(a, cfg->dtype == MOE_BF16, static_cast<hipStream_t>(stream)));
  return MOE_OK;
}

size_t moe_norm_backward_workspace_bytes(const moe_norm_cfg* cfg, int64_t T) {
  if (validate(cfg, T) != MOE_OK || T == 0) return 0;
  moe::NormArgs a{};
  return norm_carve(*cfg, T, nullptr, a);
}

int moe_norm_backward(const moe_norm_cfg* cfg, int64_t T, const void* residual, int64_t ld_residual,
                      const void* branch, int64_t ld_branch, const moe_norm_params* params, const void* du,
                      int64_t ld_du, const void* dh, int64_t ld_dh, const moe_norm_grads* grads, void* ws,
                      size_t ws_bytes, void* stream) {
  int rc = validate(cfg, T);
  if (rc != MOE_OK || T == 0) return rc;
  if (residual == nullptr || grads == nullptr || (du == nullptr && dh == nullptr)) return MOE_ERR_NULL;
  if ((rc = check_params(*cfg, params, branch != nullptr, dh != nullptr)) != MOE_OK) return rc;
  if ((grads->d_branch != nullptr && branch == nullptr) || (grads->dw_post != nullptr && params->w_post == nullptr) ||
      (grads->db_post != nullptr && params->b_post == nullptr) ||
      (grads->dw_pre != nullptr && (params->w_pre == nullptr || dh == nullptr)) ||
      (grads->db_pre != nullptr && (params->b_pre == nullptr || dh == nullptr)) ||
      (grads->dgate != nullptr && params->gate == nullptr))
    return MOE_ERR_NULL;
  const int64_t H = cfg->hidden;
  if (bad_ld(residual, ld_residual, H) || bad_ld(branch, ld_branch, H) || bad_ld(du, ld_du, H) ||
      bad_ld(dh, ld_dh, H) || bad_ld(grads->d_residual, grads->ld_d_residual, H) ||
      bad_ld(grads->d_branch, grads->ld_d_branch, H))
    return MOE_ERR_SHAPE;
  moe::NormArgs a = norm_args(*cfg, T, residual, ld_residual, branch, ld_branch, *params);
  if (bad_ws(ws, ws_bytes, norm_carve(*cfg, T, ws, a))) return MOE_ERR_WORKSPACE;
  if ((rc = check_device()) != MOE_OK) return rc;
  a.du = du;
  a.ld_du = ld_du;
  a.dh = dh;
  a.ld_dh = ld_dh;
  a.d_residual = grads->d_residual;
  a.ld_dr = grads->ld_d_residual;
  a.d_branch = grads->d_branch;
  a.ld_db = grads->ld_d_branch;
  a.dw_post = grads->dw_post;
  a.db_post = grads->db_post;
  a.dw_pre = grads->dw_pre;
  a.db_pre = grads->db_pre;
  a.dgate = grads->dgate;
  MOE_TRY(moe::launch_norm_backward(a, cfg->dtype == MOE_BF16, static_cast<hipStream_t>(stream)));
  return MOE_OK;
}

// ---------------------------------------------------------------- linear

size_t moe_linear_workspace_bytes(const moe_linear_cfg* cfg, int64_t T) {
  if (validate(cfg, T) != MOE_OK || T == 0) return 0;
  return linear_carve(*cfg, kUpTo, T, false, nullptr, nullptr, 0, nullptr, nullptr, 0).bytes;
}

int moe_linear_forward(const moe_linear_cfg* cfg, int64_t T, const void* x, int64_t ld_x, const void* w,
                       const void* bias, const void* residual, int64_t ld_residual, void* y, int64_t ld_y, void* ws,
                       size_t ws_bytes, void* stream) {
  int rc = validate(cfg, T);
  if (rc != MOE_OK || T == 0) return rc;
  if (x == nullptr || w == nullptr || y == nullptr) return MOE_ERR_NULL;
  const int K = cfg->in_dim, N = cfg->out_dim;
  if (bad_ld(x, ld_x, K) || bad_ld(residual, ld_residual, N) || bad_ld(y, ld_y, N)) return MOE_ERR_SHAPE;
  const LinearWork L = linear_carve(*cfg, kThis, T, false, ws, x, ld_x, w, nullptr, 0);
  if (bad_ws(ws, ws_bytes, L.bytes)) return MOE_ERR_WORKSPACE;
  if ((rc = check_device()) != MOE_OK) return rc;
  const bool f32 = cfg->dtype == MOE_F32;
  hipStream_t st = static_cast<hipStream_t>(stream);
  if (streams(T, f32)) {
    const moe::DenseStreamArgs a{x,    w,    nullptr,     bias, residual, y,
                                 ld_x, ld_residual, ld_y, int(T), N, K, cfg->act};
    MOE_TRY(moe::launch_dense_stream(a, f32, st));
    return MOE_OK;
  }
  Operands ops(f32);
  const Mat X = ops.add(L.x), W = ops.add(L.w);
  MOE_TRY(ops.lay_out(st));
  moe::DenseArgs g = product(T, N, K, moe::kEpiOut, f32);
  add_segments(g, f32, X, W);
  g.epi.act = cfg->act;
  g.epi.bias = bias;
  g.epi.residual = residual;
  g.epi.ld_residual = ld_residual;
  g.epi.out = y;
  g.epi.ld_out = ld_y;
  MOE_TRY(launch(g, moe::kNT, L.part, st));
  return MOE_OK;
}

size_t moe_linear_backward_workspace_bytes(const moe_linear_cfg* cfg, int64_t T) {
  if (validate(cfg, T) != MOE_OK || T == 0) return 0;
  return linear_carve(*cfg, kUpTo, T, true, nullptr, nullptr, 0, nullptr, nullptr, 0).bytes;
}

int moe_linear_backward(const moe_linear_cfg* cfg, int64_t T, const void* x, int64_t ld_x, const void* w,
                        const void* bias, const void* dy, int64_t ld_dy, void* dx, int64_t ld_dx, void* dw,
                        void* dbias, void* ws, size_t ws_bytes, void* stream) {
  int rc = validate(cfg, T);
  if (rc != MOE_OK || T == 0) return rc;
  if (x == nullptr || w == nullptr || dy == nullptr) return MOE_ERR_NULL;
  const int K = cfg->in_dim, N = cfg->out_dim;
  if (bad_ld(x, ld_x, K) || bad_ld(dy, ld_dy, N) || bad_ld(dx, ld_dx, K)) return MOE_ERR_SHAPE;
  const LinearWork L = linear_carve(*cfg, kThis, T, true, ws, x, ld_x, w, dy, ld_dy);
  if (bad_ws(ws, ws_bytes, L.bytes)) return MOE_ERR_WORKSPACE;
  if (dx == nullptr && dw == nullptr && dbias == nullptr) return MOE_OK;
  if ((rc = check_device()) != MOE_OK) return rc;
  const bool f32 = cfg->dtype == MOE_F32, plain = cfg->act == MOE_ACT_NONE;
  hipStream_t st = static_cast<hipStream_t>(stream);
  Mat X{}, W{}, DZ{};
  Operands ops(f32);
  if (!plain || dw != nullptr) X = ops.add(L.x);
  if (!plain || dx != nullptr) W = ops.add(L.w);
  if (plain && (dx != nullptr || dw != nullptr)) DZ = ops.add(L.dy);
  MOE_TRY(ops.lay_out(st));
  if (plain) {
    if (dbias != nullptr)
      MOE_TRY(moe::launch_dense_colsum(dy, f32, ld_dy, T, N, dbias, f32, L.sums, st));
  } else {
    DZ = planes_at(f32, L.dz, T, N);
    moe::DenseArgs g = product(T, N, K, moe::kEpiActBack, f32);
    add_segments(g, f32, X, W);
    g.epi.act = cfg->act;
    g.epi.bias = bias;
    g.epi.dy = dy;
    g.epi.ld_dy = ld_dy;
    g.epi.p0 = L.dz;
    stage_to(g.epi, DZ, T);
    MOE_TRY(moe::launch_dense_act_back(g, dbias, L.sums, L.part, st));
  }
  moe::DenseArgs data{};
  moe::DenseGroup weights{};
  if (dx != nullptr) {
    data = product(T, K, N, moe::kEpiOut, f32);
    add_segments(data, f32, DZ, W);
    data.epi.out = dx;
    data.epi.ld_out = ld_dx;
  }
  if (dw != nullptr) {
    weights.g[0] = product(N, K, T, moe::kEpiOut, f32);
    add_segments(weights.g[0], f32, DZ, X);
    weights.g[0].epi.out = dw;
    weights.g[0].epi.ld_out = K;
  }
  if (dx != nullptr && dw != nullptr) MOE_TRY(moe::launch_dense_gradients(data, weights, 1, L.part, st));
  else if (dx != nullptr) MOE_TRY(launch(data, moe::kNN, L.part, st));
  else if (dw != nullptr) MOE_TRY(moe::launch_dense(weights, 1, moe::kTN, L.part, st));
  return MOE_OK;
}

// ---------------------------------------------------------------- ffn

size_t moe_ffn_workspace_bytes(const moe_ffn_cfg* cfg, int64_t T) {
  if (validate(cfg, T) != MOE_OK || T == 0) return 0;
  return ffn_carve(*cfg, kUpTo, T, false, nullptr, nullptr, 0, nullptr, nullptr, nullptr, nullptr, 0).bytes;
}

int moe_ffn_forward(const moe_ffn_cfg* cfg, int64_t T, const void* x, int64_t ld_x, const void* w_gate,
                    const void* w_up, const void* w_down, const void* residual, int64_t ld_residual, void* y,
                    int64_t ld_y, void* ws, size_t ws_bytes, void* stream) {
  int rc = validate(cfg, T);
  if (rc != MOE_OK || T == 0) return rc;
  if (x == nullptr || w_gate == nullptr || w_up == nullptr || w_down == nullptr || y == nullptr) return MOE_ERR_NULL;
  const int H = cfg->hidden, I = cfg->inter;
  if (bad_ld(x, ld_x, H) || bad_ld(residual, ld_residual, H) || bad_ld(y, ld_y, H)) return MOE_ERR_SHAPE;
  const FfnWork F = ffn_carve(*cfg, kThis, T, false, ws, x, ld_x, w_gate, w_up, w_down, nullptr, 0);
  if (bad_ws(ws, ws_bytes, F.bytes)) return MOE_ERR_WORKSPACE;
  if ((rc = check_device()) != MOE_OK) return rc;
  const bool f32 = cfg->dtype == MOE_F32;
  hipStream_t st = static_cast<hipStream_t>(stream);
  if (streams(T, f32)) {
    const moe::DenseStreamArgs up{x, w_gate, w_up, nullptr, nullptr, F.mid, ld_x, 0, I, int(T), I, H, cfg->act};
    MOE_TRY(moe::launch_dense_stream(up, f32, st));
    const moe::DenseStreamArgs down{F.mid, w_down, nullptr, nullptr,     residual, y,
                                    I,     ld_residual, ld_y, int(T), H,        I, MOE_ACT_NONE};
    MOE_TRY(moe::launch_dense_stream(down, f32, st));
    return MOE_OK;
  }
  Operands ops(f32);
  const bool both = direct(F.wg) && direct(F.wu);  // the dual product reads both with one stride
  const Mat X = ops.add(F.x), WG = ops.add(F.wg, both), WU = ops.add(F.wu, both), WD = ops.add(F.wd);
  MOE_TRY(ops.lay_out(st));
  const Mat MID = planes_at(f32, F.mid, T, I);
  moe::DenseArgs g = product(T, I, H, moe::kEpiGated, f32);
  add_segments(g, f32, X, WG, &WU);
  g.epi.act = cfg->act;
  g.epi.p0 = F.mid;
  stage_to(g.epi, MID, T);
  MOE_TRY(launch(g, moe::kNT, F.part, st));
  g = product(T, H, I, moe::kEpiOut, f32);
  add_segments(g, f32, MID, WD);
  g.epi.residual = residual;
  g.epi.ld_residual = ld_residual;
  g.epi.out = y;
  g.epi.ld_out = ld_y;
  MOE_TRY(launch(g, moe::kNT, F.part, st));
  return MOE_OK;
}

size_t moe_ffn_backward_workspace_bytes(const moe_ffn_cfg* cfg, int64_t T) {
  if (validate(cfg, T) != MOE_OK || T == 0) return 0;
  return ffn_carve(*cfg, kUpTo, T, true, nullptr, nullptr, 0, nullptr, nullptr, nullptr, nullptr, 0).bytes;
}

int moe_ffn_backward(const moe_ffn_cfg* cfg, int64_t T, const void* x, int64_t ld_x, const void* w_gate,
                     const void* w_up, const void* w_down, const void* dy, int64_t ld_dy, void* dx, int64_t ld_dx,
                     void* dw_gate, void* dw_up, void* dw_down, void* ws, size_t ws_bytes, void* stream) {
  int rc = validate(cfg, T);
  if (rc != MOE_OK || T == 0) return rc;
  if (x == nullptr || w_gate == nullptr || w_up == nullptr || w_down == nullptr || dy == nullptr || dx == nullptr ||
      dw_gate == nullptr || dw_up == nullptr || dw_down == nullptr)
    return MOE_ERR_NULL;
  const int H = cfg->hidden, I = cfg->inter;
  if (bad_ld(x, ld_x, H) || bad_ld(dy, ld_dy, H) || bad_ld(dx, ld_dx, H)) return MOE_ERR_SHAPE;
  const FfnWork F = ffn_carve(*cfg, kThis, T, true, ws, x, ld_x, w_gate, w_up, w_down, dy, ld_dy);
  if (bad_ws(ws, ws_bytes, F.bytes)) return MOE_ERR_WORKSPACE;
  if ((rc = check_device()) != MOE_OK) return rc;
  const bool f32 = cfg->dtype == MOE_F32;
  hipStream_t st = static_cast<hipStream_t>(stream);
  Operands ops(f32);
  const bool both = direct(F.wg) && direct(F.wu);
  const Mat X = ops.add(F.x), WG = ops.add(F.wg, both), WU = ops.add(F.wu, both), WD = ops.add(F.wd),
            DY = ops.add(F.dy);
  MOE_TRY(ops.lay_out(st));
  const Mat MID = planes_at(f32, F.mid, T, I), DG = planes_at(f32, F.dg, T, I), DU = planes_at(f32, F.du, T, I);
  // The projections again, kept in float32: with bfloat16 the slope and the
  // product would carry a rounding of their own on top of the staged operands'.
  moe::DenseArgs g = product(T, I, H, moe::kEpiKeep, f32);
  add_segments(g, f32, X, WG, &WU);
  g.epi.g = F.g;
  g.epi.u = F.u;
  stage_to(g.epi, MID, T);
  MOE_TRY(launch(g, moe::kNT, F.part, st));
  // the middle's gradient, and from it the projections' and the middle itself
  g = product(T, I, H, moe::kEpiGatedBack, f32);
  add_segments(g, f32, DY, WD);
  g.epi.act = cfg->act;
  g.epi.g = F.g;
  g.epi.u = F.u;
  g.epi.p0 = F.dg;
  g.epi.p1 = F.du;
  g.epi.p2 = F.mid;
  stage_to(g.epi, MID, T);
  MOE_TRY(launch(g, moe::kNN, F.part, st));
  g = product(T, H, I, moe::kEpiOut, f32);
  add_segments(g, f32, DG, WG);
  add_segments(g, f32, DU, WU);
  g.epi.out = dx;
  g.epi.ld_out = ld_dx;
  const struct { const Mat &a, &b; int rows, cols; void* out; } grads[3] = {
      {DG, X, I, H, dw_gate}, {DU, X, I, H, dw_up}, {DY, MID, H, I, dw_down}};
  moe::DenseGroup group{};
  for (int i = 0; i < 3; ++i) {
    group.g[i] = product(grads[i].rows, grads[i].cols, T, moe::kEpiOut, f32);
    add_segments(group.g[i], f32, grads[i].a, grads[i].b);
    group.g[i].epi.out = grads[i].out;
    group.g[i].epi.ld_out = grads[i].cols;
  }
  MOE_TRY(moe::launch_dense_gradients(g, group, 3, F.part, st));
  return MOE_OK;
}

}  // extern "C"
