// C ABI of the operators with microscaled operands (quantisation, projections and
// the gated feed-forward block with 4-bit weights): argument checks, workspace
// layout and launch order.  The norm with a microscaled output is in block_api.cpp.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "block_checks.h"
#include "mx.h"

namespace {

using namespace moe::checks;

int check_matrix(int32_t format, int32_t dtype, int64_t rows, int32_t cols) {
  if (check_format(format) != MOE_OK || check_dtype(dtype) != MOE_OK) return MOE_ERR_DTYPE;
  return bad_rows(rows) || bad_dim(cols) ? MOE_ERR_SHAPE : MOE_OK;
}

int validate(const moe_mx_linear_cfg* c, int64_t T) {
  if (c == nullptr) return MOE_ERR_NULL;
  if (check_dtype(c->dtype) != MOE_OK || check_format(c->format) != MOE_OK) return MOE_ERR_DTYPE;
  if (bad_dim(c->in_dim) || bad_dim(c->out_dim) || bad_rows(T)) return MOE_ERR_SHAPE;
  if (c->act < MOE_ACT_NONE || c->act > MOE_ACT_GELU) return MOE_ERR_SHAPE;
  return MOE_OK;
}

int validate(const moe_mx_ffn_cfg* c, int64_t T) {
  if (c == nullptr) return MOE_ERR_NULL;
  if (check_dtype(c->dtype) != MOE_OK || check_format(c->format) != MOE_OK) return MOE_ERR_DTYPE;
  if (bad_dim(c->hidden) || bad_dim(c->inter) || bad_rows(T)) return MOE_ERR_SHAPE;
  if (c->act != MOE_ACT_RELU && c->act != MOE_ACT_SILU && c->act != MOE_ACT_GELU) return MOE_ERR_SHAPE;
  return MOE_OK;
}

// Room for the parts of split contractions: of T tokens' and every smaller batch's.
// Few tokens have none: nothing but a size that is not 0, which a query has for
// what is invalid, and a call asks for what its query said.
struct LinearWork {
  float* part;
  size_t bytes;
};
LinearWork linear_carve(const moe_mx_linear_cfg& c, int64_t T, void* ws) {
  Carver v{static_cast<char*>(ws)};
  LinearWork L{};
  L.part = v.take<float>(T > moe::kMxStreamTokens ? moe::mx_part_bytes(T, c.out_dim, false) : 1);
  L.bytes = v.used;
  return L;
}

// Few tokens: whether the middle is quantised by a launch of its own, and not by the
// down projection's workgroups, each for itself as it reads it.  That launch costs 3
// us, as much as a wave's quantising of four steps (hidden 2048, a call, one and 16
// tokens: inter 4096 13.3 and 16.9 us inside, 16.4 and 16.5 apart; 7168 17.2 and
// 26.7, 16.4 and 19.6).
bool quantises_apart(int inter) { return moe::mx_steps(inter) > 32; }

struct FfnWork {
  float* mid;               // few tokens: the middle
  uint8_t *codes, *scales;  // and quantised
  float* part;
  size_t bytes;
};
FfnWork ffn_carve(const moe_mx_ffn_cfg& c, int64_t T, void* ws) {
  Carver v{static_cast<char*>(ws)};
  FfnWork F{};
  const bool few = T <= moe::kMxStreamTokens;
  const size_t mid = size_t(std::min<int64_t>(T, moe::kMxStreamTokens)) * size_t(moe::mx_steps(c.inter)) * 128 * sizeof(float);
  F.codes = v.take<uint8_t>(moe_mx_code_bytes(c.format, T, c.inter));
  F.scales = v.take<uint8_t>(moe_mx_scale_bytes(T, c.inter));
  const size_t parts = std::max(moe::mx_part_bytes(T, c.inter, true), moe::mx_part_bytes(T, c.hidden, false));
  F.part = v.take<float>(few ? mid : std::max(mid, parts));
  F.mid = F.part;
  F.bytes = v.used;
  return F;
}

moe::MxArgs product(int64_t T, int N, int K, const moe_mx* x, const moe_mx* w, int act, bool f32) {
  moe::MxArgs a{};
  a.x = x->codes;
  a.sx = x->scales;
  a.w = w->codes;
  a.sw = w->scales;
  a.T = T;
  a.N = N;
  a.steps = int(moe::mx_steps(K));
  a.exact = f32;
  a.epi.mode = moe::kEpiOut;
  a.epi.act = act;
  a.epi.f32 = f32;
  a.epi.M = T;
  a.epi.N = N;
  return a;
}
void output(moe::MxArgs& a, const void* bias, const void* residual, int64_t ld_residual, void* y, int64_t ld_y) {
  a.epi.bias = bias;
  a.epi.residual = residual;
  a.epi.ld_residual = ld_residual;
  a.epi.out = y;
  a.epi.ld_out = ld_y;
}

int check_operands(const moe_mx* const* m, int count) {
  for (int i = 0; i < count; ++i)
    if (m[i] == nullptr || m[i]->codes == nullptr || m[i]->scales == nullptr) return MOE_ERR_NULL;
  for (int i = 0; i < count; ++i)
    if (bad_mx(m[i]->codes, m[i]->scales)) return MOE_ERR_SHAPE;
  return MOE_OK;
}

}  // namespace

extern "C" {

size_t moe_mx_code_bytes(int32_t format, int64_t rows, int32_t cols) {
  if (check_matrix(format, MOE_F32, rows, cols) != MOE_OK) return 0;
  return size_t(rows) * size_t(moe::mx_steps(cols)) * size_t(moe::mx_step_bytes(format));
}

size_t moe_mx_scale_bytes(int64_t rows, int32_t cols) {
  if (check_matrix(MOE_MX_E4M3, MOE_F32, rows, cols) != MOE_OK) return 0;
  return size_t(rows) * size_t(moe::mx_steps(cols)) * 4;
}

int moe_mx_quantize(int32_t format, int32_t dtype, int64_t rows, int32_t cols, const void* x, int64_t ld_x,
                    uint8_t* codes, uint8_t* scales, void* stream) {
  int rc = check_matrix(format, dtype, rows, cols);
  if (rc != MOE_OK || rows == 0) return rc;
  if (x == nullptr || codes == nullptr || scales == nullptr) return MOE_ERR_NULL;
  if (bad_ld(x, ld_x, cols) || bad_mx(codes, scales)) return MOE_ERR_SHAPE;
  if ((rc = check_device()) != MOE_OK) return rc;
  MOE_TRY(moe::launch_mx_quantize(format, dtype == MOE_F32, x, ld_x, rows, cols, codes, scales,
                                  static_cast<hipStream_t>(stream)));
  return MOE_OK;
}

int moe_mx_dequantize(int32_t format, int32_t dtype, int64_t rows, int32_t cols, const uint8_t* codes,
                      const uint8_t* scales, void* y, int64_t ld_y, void* stream) {
  int rc = check_matrix(format, dtype, rows, cols);
  if (rc != MOE_OK || rows == 0) return rc;
  if (y == nullptr || codes == nullptr || scales == nullptr) return MOE_ERR_NULL;
  if (bad_ld(y, ld_y, cols) || bad_mx(codes, scales)) return MOE_ERR_SHAPE;
  if ((rc = check_device()) != MOE_OK) return rc;
  MOE_TRY(moe::launch_mx_dequantize(format, dtype == MOE_F32, codes, scales, rows, cols, y, ld_y,
                                    static_cast<hipStream_t>(stream)));
  return MOE_OK;
}

// ---------------------------------------------------------------- linear

size_t moe_mx_linear_workspace_bytes(const moe_mx_linear_cfg* cfg, int64_t T) {
  if (validate(cfg, T) != MOE_OK || T == 0) return 0;
  return linear_carve(*cfg, T, nullptr).bytes;
}

int moe_mx_linear_forward(const moe_mx_linear_cfg* cfg, int64_t T, const moe_mx* x, const moe_mx* w, const void* bias,
                          const void* residual, int64_t ld_residual, void* y, int64_t ld_y, void* ws, size_t ws_bytes,
                          void* stream) {
  int rc = validate(cfg, T);
  if (rc != MOE_OK || T == 0) return rc;
  const moe_mx* const m[] = {x, w};
  if (y == nullptr) return MOE_ERR_NULL;
  if ((rc = check_operands(m, 2)) != MOE_OK) return rc;
  const int N = cfg->out_dim;
  if (bad_ld(residual, ld_residual, N) || bad_ld(y, ld_y, N)) return MOE_ERR_SHAPE;
  const LinearWork L = linear_carve(*cfg, T, ws);
  if (bad_ws(ws, ws_bytes, L.bytes)) return MOE_ERR_WORKSPACE;
  if ((rc = check_device()) != MOE_OK) return rc;
  moe::MxArgs a = product(T, N, cfg->in_dim, x, w, cfg->act, cfg->dtype == MOE_F32);
  output(a, bias, residual, ld_residual, y, ld_y);
  hipStream_t st = static_cast<hipStream_t>(stream);
  MOE_TRY(T <= moe::kMxStreamTokens ? moe::launch_mx_stream(a, cfg->format, st)
                                    : moe::launch_mx_gemm(a, cfg->format, L.part, st));
  return MOE_OK;
}

// ---------------------------------------------------------------- ffn

size_t moe_mx_ffn_workspace_bytes(const moe_mx_ffn_cfg* cfg, int64_t T) {
  if (validate(cfg, T) != MOE_OK || T == 0) return 0;
  return ffn_carve(*cfg, T, nullptr).bytes;
}

int moe_mx_ffn_forward(const moe_mx_ffn_cfg* cfg, int64_t T, const moe_mx* x, const moe_mx* w_gate, const moe_mx* w_up,
                       const moe_mx* w_down, const void* residual, int64_t ld_residual, void* y, int64_t ld_y, void* ws,
                       size_t ws_bytes, void* stream) {
  int rc = validate(cfg, T);
  if (rc != MOE_OK || T == 0) return rc;
  const moe_mx* const m[] = {x, w_gate, w_up, w_down};
  if (y == nullptr) return MOE_ERR_NULL;
  if ((rc = check_operands(m, 4)) != MOE_OK) return rc;
  const int H = cfg->hidden, I = cfg->inter;
  if (bad_ld(residual, ld_residual, H) || bad_ld(y, ld_y, H)) return MOE_ERR_SHAPE;
  const FfnWork F = ffn_carve(*cfg, T, ws);
  if (bad_ws(ws, ws_bytes, F.bytes)) return MOE_ERR_WORKSPACE;
  if ((rc = check_device()) != MOE_OK) return rc;
  hipStream_t st = static_cast<hipStream_t>(stream);
  moe::MxArgs up = product(T, I, H, x, w_gate, cfg->act, cfg->dtype == MOE_F32);
  up.w2 = w_up->codes;
  up.sw2 = w_up->scales;
  const bool few = T <= moe::kMxStreamTokens;
  const moe_mx mid{F.codes, F.scales};
  moe::MxArgs down = product(T, H, I, &mid, w_down, MOE_ACT_NONE, cfg->dtype == MOE_F32);
  output(down, nullptr, residual, ld_residual, y, ld_y);
  if (few) {
    up.mid = F.mid;
    MOE_TRY(moe::launch_mx_stream(up, cfg->format, st));
    if (quantises_apart(I))
      MOE_TRY(moe::launch_mx_quantize(cfg->format, true, F.mid, moe::mx_steps(I) * 128, T, I, F.codes, F.scales, st));
    else
      down.middle = F.mid;
    MOE_TRY(moe::launch_mx_stream(down, cfg->format, st));
  } else {
    up.codes = F.codes;
    up.scales = F.scales;
    MOE_TRY(moe::launch_mx_gemm(up, cfg->format, F.part, st));
    MOE_TRY(moe::launch_mx_gemm(down, cfg->format, F.part, st));
  }
  return MOE_OK;
}

}  // extern "C"
