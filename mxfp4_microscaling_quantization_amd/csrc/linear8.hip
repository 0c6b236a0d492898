// The 8-bit linear layer: quantizers and products composed.
//   Y  = Q(X) Q(W)^T             Q(X): 1x128 blocks, Q(W): 128x128 tiles
//   dX = Q(dY) Q(W)              Q(dY): 1x128 blocks; Q(W) in its second layout, the same values
//   dW = Q(dY)^T Q(Q(X))         128x1 blocks along the rows of dY and of what the forward kept of X
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "mx_host8.h"

namespace mx {

static int64_t round256(int64_t n) { return (n + 255) / 256 * 256; }

// The backward's operands in its workspace: dY by rows and by columns, X by columns, the
// products' partial sums.
struct Linear8Layout {
  int64_t ld_n, ld_m, ls_n, ls_m;
  int64_t dy, dys, dyt, dyts, xt, xts, part, total;
};
static Linear8Layout linear8_layout(int64_t M, int64_t N, int64_t K) {
  Linear8Layout l;
  l.ld_n = round16(N), l.ls_n = scale8_pitch(N);
  l.ld_m = round16(M), l.ls_m = scale8_pitch(M);
  int64_t at = 0;
  auto take = [&](int64_t bytes) {
    const int64_t p = at;
    at += round256(bytes);
    return p;
  };
  l.dy = take(M * l.ld_n), l.dys = take(M * l.ls_n);
  l.dyt = take(N * l.ld_m), l.dyts = take(N * l.ls_m);
  l.xt = take(K * l.ld_m), l.xts = take(K * l.ls_m);
  l.part = take((int64_t)gemm8_two_workspace(M, K, N, N, K, M));
  l.total = at;
  return l;
}

static bool linear8_shape(int64_t M, int64_t N, int64_t K) {
  return M >= 0 && N >= 0 && K >= 0 && M <= kMaxAxis8 && N <= kMaxAxis8 && K <= kMaxAxis8;
}

}  // namespace mx

using namespace mx;

extern "C" size_t mx_linear8_fwd_workspace_size(int64_t M, int64_t N, int64_t K) {
  return linear8_shape(M, N, K) && M && N && K ? gemm8_workspace(M, N, K) : 0;
}

extern "C" int mx_linear8_fwd(const void* x, int x_dtype, int64_t ldx, const void* w, int w_dtype, int64_t ldw,
                              int64_t M, int64_t N, int64_t K, void* y, int y_dtype, int64_t ldy,
                              uint8_t* xq_codes, uint8_t* xq_scales, uint8_t* wq_codes, uint8_t* wq_scales,
                              uint8_t* wt_codes, uint8_t* wt_scales, void* workspace, size_t workspace_bytes,
                              void* stream) {
  MX_REQUIRE(float_type(x_dtype) && float_type(y_dtype) && (!w || float_type(w_dtype)), MX_ERR_ENUM);
  MX_REQUIRE(linear8_shape(M, N, K) && ldx >= K && ldy >= N && (!w || ldw >= K), MX_ERR_SHAPE);
  if (M == 0 && (!w || N == 0 || K == 0)) return MX_OK;
  if (N == 0 && K == 0) return MX_OK;
  if (M && N) {
    MX_REQUIRE(y, MX_ERR_NULL);
    MX_REQUIRE(aligned16(y), MX_ERR_ALIGN);
  }
  if (M && K) {
    MX_REQUIRE(x && xq_codes && xq_scales, MX_ERR_NULL);
    MX_REQUIRE(aligned16(x) && aligned16(xq_codes) && aligned16(xq_scales), MX_ERR_ALIGN);
  }
  if (N && K) {
    MX_REQUIRE(wq_codes && wq_scales && !wt_codes == !wt_scales, MX_ERR_NULL);
    MX_REQUIRE(aligned16(w) && aligned16(wq_codes) && aligned16(wq_scales) && aligned16(wt_codes) &&
                   aligned16(wt_scales), MX_ERR_ALIGN);
  }
  const size_t need = mx_linear8_fwd_workspace_size(M, N, K);
  if (need) {
    MX_REQUIRE(workspace && workspace_bytes >= need, MX_ERR_WORKSPACE);
    MX_REQUIRE(aligned16(workspace), MX_ERR_ALIGN);
  }
  const hipStream_t st = as_stream(stream);
  const int64_t ldk = round16(K), lsk = scale8_pitch(K);
  int s;
  if (w && M && N && K) {
    s = quant8_forward_impl(x, x_dtype, ldx, M, w, w_dtype, ldw, N, K, xq_codes, xq_scales, wq_codes, wq_scales,
                            wt_codes, wt_scales, st);
  } else {
    s = quant8_row_impl(x, x_dtype, ldx, M, K, xq_codes, ldk, xq_scales, lsk, st);
    if (s == MX_OK && w)
      s = quant8_tile_impl(w, w_dtype, ldw, N, K, true, wq_codes, ldk, wq_scales, lsk, wt_codes, round16(N), wt_scales,
                           scale8_pitch(N), st);
  }
  if (s != MX_OK) return s;
  return gemm8_impl({xq_codes, xq_scales, wq_codes, wq_scales, ldk, lsk, ldk, lsk, M, N, K, 1.0f, y, y_dtype, ldy},
                    workspace, st);
}

extern "C" size_t mx_linear8_bwd_workspace_size(int64_t M, int64_t N, int64_t K) {
  return linear8_shape(M, N, K) && M && N && K ? (size_t)linear8_layout(M, N, K).total : 0;
}

extern "C" int mx_linear8_bwd(const void* dy, int dy_dtype, int64_t lddy, int64_t M, int64_t N, int64_t K,
                              const uint8_t* xq_codes, const uint8_t* xq_scales, const uint8_t* wt_codes,
                              const uint8_t* wt_scales, void* dx, int dx_dtype, int64_t lddx, float* dw,
                              int64_t lddw, void* workspace, size_t workspace_bytes, void* stream) {
  MX_REQUIRE(float_type(dy_dtype) && float_type(dx_dtype), MX_ERR_ENUM);
  MX_REQUIRE(linear8_shape(M, N, K) && lddy >= N && lddx >= K && lddw >= K, MX_ERR_SHAPE);
  if (K == 0 || (M == 0 && N == 0)) return MX_OK;
  const hipStream_t st = as_stream(stream);
  MX_REQUIRE((M == 0 || dx) && (N == 0 || dw), MX_ERR_NULL);
  MX_REQUIRE(aligned16(dx) && aligned16(dw), MX_ERR_ALIGN);
  if (M == 0 || N == 0) {  // an empty contraction: the other gradient has no entries
    const Product8 none = {nullptr, nullptr, nullptr, nullptr, 0, 0, 0, 0, M ? M : N, K, 0, 1.0f, M ? dx : dw,
                           M ? dx_dtype : MX_F32, M ? lddx : lddw};
    return gemm8_impl(none, nullptr, st);
  }
  MX_REQUIRE(dy && xq_codes && xq_scales && wt_codes && wt_scales, MX_ERR_NULL);
  MX_REQUIRE(aligned16(dy) && aligned16(xq_codes) && aligned16(xq_scales) && aligned16(wt_codes) &&
                 aligned16(wt_scales), MX_ERR_ALIGN);
  const Linear8Layout l = linear8_layout(M, N, K);
  MX_REQUIRE(workspace && workspace_bytes >= (size_t)l.total, MX_ERR_WORKSPACE);
  MX_REQUIRE(aligned16(workspace), MX_ERR_ALIGN);
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  int s = quant8_backward_impl(dy, dy_dtype, lddy, M, N, xq_codes, xq_scales, K, ws + l.dy, ws + l.dys, ws + l.dyt,
                               ws + l.dyts, ws + l.xt, ws + l.xts, st);
  if (s != MX_OK) return s;
  return gemm8_two_impl({ws + l.dy, ws + l.dys, wt_codes, wt_scales, l.ld_n, l.ls_n, round16(N), scale8_pitch(N), M, K, N, 1.0f,
                         dx, dx_dtype, lddx},
                        {ws + l.dyt, ws + l.dyts, ws + l.xt, ws + l.xts, l.ld_m, l.ls_m, l.ld_m, l.ls_m, N, K, M, 1.0f, dw,
                         MX_F32, lddw},
                        ws + l.part, st);
}
