// Host-side layout of the 8-bit matrices, shared by the quantizers, products and layers.
#pragma once

#include "mx_host.h"

namespace mx {

inline int64_t round16(int64_t n) { return (n + 15) / 16 * 16; }
inline int64_t blocks8(int64_t n) { return cdiv(n, 128); }
inline int64_t scale8_pitch(int64_t n) { return cdiv(n, 512) * 4; }  // whole dwords of bytes
inline bool float_type(int t) { return t == MX_F32 || t == MX_BF16; }
constexpr int64_t kMax8 = (int64_t)1 << 31;       // rows and columns are below this
constexpr int64_t kMaxAxis8 = (int64_t)1 << 23;   // contraction axes and pitches: 256 rows span less than 2^31 bytes

// A [rows, cols] 8-bit matrix at these pitches.  A product keeps offsets within 256 rows of codes and of scales in
// 32 bits.
inline bool matrix8(int64_t cols, int64_t ld, int64_t scale_ld) {
  return ld >= round16(cols) && ld % 16 == 0 && ld <= kMaxAxis8 && scale_ld >= scale8_pitch(cols) &&
         scale_ld % 4 == 0 && scale_ld <= kMaxAxis8;
}

int quant8_row_impl(const void* x, int dtype, int64_t ldx, int64_t rows, int64_t cols, uint8_t* codes,
                    int64_t ld, uint8_t* scales, int64_t scale_ld, hipStream_t st);
// Blocks of 128x128 (tile) or 1x128 and 128x1 from one read; either output may be NULL.
int quant8_tile_impl(const void* x, int dtype, int64_t ldx, int64_t rows, int64_t cols, bool tile,
                     uint8_t* codes, int64_t ld, uint8_t* scales, int64_t scale_ld, uint8_t* codes_t,
                     int64_t ld_t, uint8_t* scales_t, int64_t scale_ld_t, hipStream_t st);
int requant8_impl(const uint8_t* codes, int64_t ld, const uint8_t* scales, int64_t scale_ld,
                  int64_t rows, int64_t cols, uint8_t* codes_t, int64_t ld_t, uint8_t* scales_t,
                  int64_t scale_ld_t, hipStream_t st);
// The 8-bit linear layer's operands, each pair in one launch; M, N, K > 0.
// Forward: x [M, K] in 1x128 blocks, w [N, K] in tiles (wt: its transpose, or NULL).
int quant8_forward_impl(const void* x, int x_dtype, int64_t ldx, int64_t M, const void* w, int w_dtype,
                        int64_t ldw, int64_t N, int64_t K, uint8_t* xq, uint8_t* xs, uint8_t* wq, uint8_t* ws,
                        uint8_t* wt, uint8_t* wts, hipStream_t st);
// Backward: dy [M, N] by rows (q, s) and by columns (qt, qts), the 8-bit x [M, K] by columns (xt, xts).
int quant8_backward_impl(const void* dy, int dtype, int64_t lddy, int64_t M, int64_t N, const uint8_t* xq,
                         const uint8_t* xs, int64_t K, uint8_t* q, uint8_t* s, uint8_t* qt, uint8_t* qts,
                         uint8_t* xt, uint8_t* xts, hipStream_t st);
size_t gemm8_workspace(int64_t M, int64_t N, int64_t K);
struct Product8 {  // c = alpha a b^T
  const uint8_t *a, *sa, *b, *sb;
  int64_t lda, lsa, ldb, lsb, M, N, K;
  float alpha;
  void* c;
  int c_dtype;
  int64_t ldc;
};
int gemm8_impl(const Product8& p, void* workspace, hipStream_t st);
// Two products (w's C is float32), in one launch where both take tiles of 128; M, N, K > 0.
size_t gemm8_two_workspace(int64_t Mx, int64_t Nx, int64_t Kx, int64_t Mw, int64_t Nw, int64_t Kw);
int gemm8_two_impl(const Product8& x, const Product8& w, void* workspace, hipStream_t st);

}  // namespace mx
