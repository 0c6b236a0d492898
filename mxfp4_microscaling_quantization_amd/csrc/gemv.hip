// Products of a few rows of unquantized activations with packed MXFP4 weights:
//   y[m][n] = alpha sum_k x[m][k] deq(W)[n][k]
// -- the single-token (decode) form of a layer whose weights are kept packed,
// and the same per expert of a mixture-of-experts layer, with the routed rows'
// ranges and sources read on the device.
//
// What bounds it: the weights are read once, 17/32 byte each, and every value
// meets only M rows of x, so for few rows HBM (or the latency of one pass over
// it) is the bound.  The products run on V_MFMA_F32_16X16X32_BF16 with 16 weight
// rows as one operand and up to 16 rows of x as the other: E2M1 values times a
// power of two are exact in bf16 (one conversion instruction per two codes), the
// products are exact in float32 and the sums are float32.  A bf16 x goes in as it
// is; a float32 x is split exactly into three bf16 terms (8 significant bits
// each, by truncation), one MFMA each.
//
// Lane layout of the MFMA operands: lane l holds row l & 15 and the 8 consecutive
// contraction values 8 (l >> 4) .. + 7.  The contraction may run in any order as
// long as both operands agree, so in a step of 128 values lane group g = l >> 4
// takes the step's block g (32 consecutive values): one 16-byte load of codes and
// one scale byte per lane feed four MFMAs, the j-th with values 8j .. 8j+7 of the
// block.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "mx_device.h"
#include "mx_host.h"

namespace mx {

typedef __bf16 v8bf __attribute__((ext_vector_type(8)));
typedef __bf16 v2bf __attribute__((ext_vector_type(2)));
typedef float v4f __attribute__((ext_vector_type(4)));

struct GemvArgs {
  const void* x;
  int64_t ldx, x_rows;
  const uint8_t* codes;
  const uint8_t* scales;
  int64_t scale_ld;
  const int64_t* offs;  // grouped: device offsets [groups + 1]
  const int32_t* src;   // grouped: slot of each row, or NULL
  int64_t M, N;         // M: rows of y
  int K, top_k, groups, y_bf16;
  float alpha;
  void* y;
  int64_t ldy, ntiles, mtiles;
};

// 8 codes (element i in nibble i) under a block scale, as bf16.
__device__ __forceinline__ v8bf decode8_bf16(uint32_t w, float scale) {
  const v2bf a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 0);
  const v2bf b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 1);
  const v2bf c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 2);
  const v2bf d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 3);
  v8bf v;
  v[0] = a.x; v[1] = a.y; v[2] = b.x; v[3] = b.y;
  v[4] = c.x; v[5] = c.y; v[6] = d.x; v[7] = d.y;
  return v;
}

// The contraction values a lane feeds one MFMA: 8 values of x as TERMS bf16 operands.
template <typename T>
struct XTerms;
template <>
struct XTerms<uint16_t> {
  static constexpr int kTerms = 1;
  static __device__ __forceinline__ void make(const uint32_t w[4], v8bf t[1]) {
    t[0] = __builtin_bit_cast(v8bf, make_uint4(w[0], w[1], w[2], w[3]));
  }
};
template <>
struct XTerms<float> {
  static constexpr int kTerms = 3;
  // Upper halves of two floats as a bf16 pair.
  static __device__ __forceinline__ uint32_t tops(float a, float b) {
    return __builtin_amdgcn_perm(__float_as_uint(b), __float_as_uint(a), 0x07060302u);
  }
  static __device__ __forceinline__ float top(float a) {
    return __uint_as_float(__float_as_uint(a) & 0xFFFF0000u);
  }
  static __device__ __forceinline__ void make(const uint32_t w[8], v8bf t[3]) {
    uint32_t o[3][4];
#pragma unroll
    for (int p = 0; p < 4; ++p) {
      float a[2], b[2], c[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const uint32_t u = w[2 * p + i];
        const bool nan = (u & 0x7FFFFFFFu) > 0x7F800000u, inf = (u & 0x7FFFFFFFu) == 0x7F800000u;
        a[i] = __uint_as_float(nan ? 0x7FC00000u : u);  // a NaN with only low bits stays a NaN
        b[i] = inf ? 0.0f : a[i] - top(a[i]);           // exact: the low 16 significant bits
        c[i] = b[i] - top(b[i]);                        // exact: the low 8
      }
      o[0][p] = tops(a[0], a[1]);
      o[1][p] = tops(b[0], b[1]);
      o[2][p] = tops(c[0], c[1]);
    }
#pragma unroll
    for (int k = 0; k < 3; ++k)
      t[k] = __builtin_bit_cast(v8bf, make_uint4(o[k][0], o[k][1], o[k][2], o[k][3]));
  }
};

// 8 values of x, raw; `wide`: on 16 bytes.
template <typename T, bool WIDE>
__device__ __forceinline__ void load_x8(const T* p, uint32_t* w) {
  constexpr int W = 2 * sizeof(T);
  if constexpr (WIDE) {
#pragma unroll
    for (int i = 0; i < W / 4; ++i) {
      const uint4 u = reinterpret_cast<const uint4*>(p)[i];
      w[4 * i] = u.x; w[4 * i + 1] = u.y; w[4 * i + 2] = u.z; w[4 * i + 3] = u.w;
    }
  } else if constexpr (sizeof(T) == 4) {
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = __float_as_uint(p[i]);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = p[2 * i] | (uint32_t)p[2 * i + 1] << 16;
  }
}

// A workgroup of W waves computes 16 NT columns of y (weight rows) for MT tiles of
// 16 rows: the waves split the contraction (wave w takes steps w, w + W, ...), their
// sums meet in LDS and are added in wave order.
template <typename T, int MT, int NT, int W, bool GROUPED, bool WIDE>
__global__ __launch_bounds__(64 * W) void k_gemv(const GemvArgs a) {
  constexpr int X = XTerms<T>::kTerms;
  constexpr int XW = 2 * sizeof(T);  // words of 8 values of x
  __shared__ v4f s_part[W][MT * NT][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int r16 = lane & 15, g = lane >> 4;
  const int nblk = a.K / 32, steps = (nblk + 3) / 4;
  const int64_t kbytes = a.K / 2;
  const T* const x = static_cast<const T*>(a.x);

  for (int64_t tile = blockIdx.x; tile < a.ntiles * a.mtiles; tile += gridDim.x) {
    const int64_t n0 = (tile % a.ntiles) * (16 * NT);
    int64_t row0 = tile / a.ntiles, row1;
    const uint8_t* codes = a.codes;
    const uint8_t* scales = a.scales;
    if constexpr (GROUPED) {
      // row0 counts the groups that hold rows
      int grp = -1;
      int64_t left = row0;
      for (int e = 0; e < a.groups; ++e) {
        if (a.offs[e + 1] > a.offs[e] && left-- == 0) {
          grp = e;
          break;
        }
      }
      if (grp < 0) break;
      row0 = max<int64_t>(a.offs[grp], 0);
      row1 = min<int64_t>(a.offs[grp + 1], a.M);
      codes += grp * a.N * kbytes;
      scales += grp * a.N * a.scale_ld;
    } else {
      row0 *= 16 * MT;
      row1 = min<int64_t>(row0 + 16 * MT, a.M);
    }
    const uint8_t* wc[NT];
    const uint8_t* ws[NT];
#pragma unroll
    for (int i = 0; i < NT; ++i) {
      const int64_t n = min<int64_t>(n0 + 16 * i + r16, a.N - 1);
      wc[i] = codes + n * kbytes;
      ws[i] = scales + n * a.scale_ld;
    }
    for (int64_t m0 = row0; m0 < row1; m0 += 16 * MT) {
      const T* xr[MT];
#pragma unroll
      for (int i = 0; i < MT; ++i) {
        int64_t r = min<int64_t>(m0 + 16 * i + r16, row1 - 1);
        if constexpr (GROUPED) {
          if (a.src) r = a.src[r] / a.top_k;
          if (r < 0 || r >= a.x_rows) r = 0;  // not stored below
        }
        xr[i] = x + r * a.ldx;
      }
      v4f acc[MT][NT];
#pragma unroll
      for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int j = 0; j < NT; ++j) acc[i][j] = v4f{0.0f, 0.0f, 0.0f, 0.0f};

      for (int s = wave; s < steps; s += W) {
        const int blk = 4 * s + g;
        const bool in = blk < nblk;
        const int b = in ? blk : 0;  // lanes past the last block read block 0 and put in zeros
        uint4 c[NT];
        uint32_t sc[NT];
#pragma unroll
        for (int i = 0; i < NT; ++i) {
          c[i] = *reinterpret_cast<const uint4*>(wc[i] + (int64_t)b * 16);
          sc[i] = ws[i][b];
        }
        uint32_t xw[MT][4][XW];
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j) load_x8<T, WIDE>(xr[i] + (int64_t)b * 32 + 8 * j, xw[i][j]);
        if (4 * s + 4 > nblk) {
#pragma unroll
          for (int i = 0; i < NT; ++i) {
            if (!in) {
              c[i] = make_uint4(0, 0, 0, 0);
              sc[i] = 127;
            }
          }
#pragma unroll
          for (int i = 0; i < MT; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j)
#pragma unroll
              for (int k = 0; k < XW; ++k) xw[i][j][k] = in ? xw[i][j][k] : 0u;
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          v8bf xt[MT][X];
#pragma unroll
          for (int i = 0; i < MT; ++i) XTerms<T>::make(xw[i][j], xt[i]);
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            const uint32_t w = j == 0 ? c[n].x : j == 1 ? c[n].y : j == 2 ? c[n].z : c[n].w;
            const v8bf wv = decode8_bf16(w, scale_of(sc[n]));
#pragma unroll
            for (int i = 0; i < MT; ++i)
#pragma unroll
              for (int k = X - 1; k >= 0; --k)
                acc[i][n] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(wv, xt[i][k], acc[i][n], 0, 0, 0);
          }
        }
      }
#pragma unroll
      for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int j = 0; j < NT; ++j) s_part[wave][i * NT + j][lane] = acc[i][j];
      __syncthreads();
      // lane (g, m) of tile (i, j) holds y[m0 + 16 i + m][n0 + 16 j + 4 g .. + 3]
      for (int o = threadIdx.x; o < MT * NT * 64; o += 64 * W) {
        const int og = o & 3, oj = (o >> 2) % NT, om = (o >> 2) / NT % 16, oi = o / (64 * NT);
        v4f sum = s_part[0][oi * NT + oj][og * 16 + om];
#pragma unroll
        for (int w = 1; w < W; ++w) sum += s_part[w][oi * NT + oj][og * 16 + om];
        const int64_t m = m0 + 16 * oi + om, n = n0 + 16 * oj + 4 * og;
        bool real = m < row1;
        if constexpr (GROUPED) {
          if (real) {
            const int64_t r = a.src ? a.src[m] / a.top_k : m;
            real = r >= 0 && r < a.x_rows && !(a.src && a.src[m] < 0);
          }
        }
        if (real) {
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            if (n + k < a.N) {
              const float v = a.alpha * sum[k];
              if (a.y_bf16) static_cast<uint16_t*>(a.y)[m * a.ldy + n + k] = (uint16_t)f32_to_bf16_rne(v);
              else static_cast<float*>(a.y)[m * a.ldy + n + k] = v;
            }
          }
        }
      }
      __syncthreads();
    }
  }
}

template <typename T, int MT, bool GROUPED, bool WIDE>
static int gemv_launch(GemvArgs a, int64_t mtiles, hipStream_t st) {
  constexpr int NT = 4, W = MT == 4 ? 4 : 8;
  a.ntiles = cdiv(a.N, 16 * NT);
  a.mtiles = mtiles;
  const unsigned grid = (unsigned)hmin(a.ntiles * mtiles, 1 << 20);
  k_gemv<T, MT, NT, W, GROUPED, WIDE><<<grid, 64 * W, 0, st>>>(a);
  return launch_status();
}

template <typename T, bool GROUPED, bool WIDE>
static int gemv_rows(const GemvArgs& a, int64_t tile_rows, int64_t groups, hipStream_t st) {
  if (tile_rows <= 16) return gemv_launch<T, 1, GROUPED, WIDE>(a, GROUPED ? groups : cdiv(a.M, 16), st);
  if (tile_rows <= 32) return gemv_launch<T, 2, GROUPED, WIDE>(a, GROUPED ? groups : cdiv(a.M, 32), st);
  return gemv_launch<T, 4, GROUPED, WIDE>(a, GROUPED ? groups : cdiv(a.M, 64), st);
}

template <bool GROUPED>
static int gemv_any(const GemvArgs& a, int x_dtype, int64_t tile_rows, int64_t groups, hipStream_t st) {
  const bool wide = a.ldx * (x_dtype == MX_BF16 ? 2 : 4) % 16 == 0;
  if (x_dtype == MX_BF16)
    return wide ? gemv_rows<uint16_t, GROUPED, true>(a, tile_rows, groups, st)
                : gemv_rows<uint16_t, GROUPED, false>(a, tile_rows, groups, st);
  return wide ? gemv_rows<float, GROUPED, true>(a, tile_rows, groups, st)
              : gemv_rows<float, GROUPED, false>(a, tile_rows, groups, st);
}

static int gemv_check(const void* x, int x_dtype, int64_t ldx, const uint8_t* w_codes,
                      const uint8_t* w_scales, int64_t w_scale_ld, int64_t M, int64_t N, int64_t K,
                      const void* y, int y_dtype, int64_t ldy) {
  constexpr int64_t kMax31 = (int64_t)1 << 31;
  MX_REQUIRE((x_dtype == MX_F32 || x_dtype == MX_BF16) && (y_dtype == MX_F32 || y_dtype == MX_BF16),
             MX_ERR_ENUM);
  MX_REQUIRE(M >= 0 && M < kMax31 && N >= 0 && N < kMax31 && K >= 0 && K < kMax31 && K % 32 == 0 &&
                 ldx >= K && ldy >= N && w_scale_ld >= K / 32, MX_ERR_SHAPE);
  if (M == 0 || N == 0) return MX_OK;
  MX_REQUIRE(y, MX_ERR_NULL);
  if (K) MX_REQUIRE(x && w_codes && w_scales, MX_ERR_NULL);
  MX_REQUIRE(aligned16(x) && aligned16(w_codes) && aligned16(w_scales) && aligned16(y), MX_ERR_ALIGN);
  return MX_OK;
}

}  // namespace mx

using namespace mx;

extern "C" int mx_gemv(const void* x, int x_dtype, int64_t ldx, const uint8_t* w_codes,
                       const uint8_t* w_scales, int64_t w_scale_ld, int64_t M, int64_t N, int64_t K,
                       float alpha, void* y, int y_dtype, int64_t ldy, void* stream) {
  const int bad = gemv_check(x, x_dtype, ldx, w_codes, w_scales, w_scale_ld, M, N, K, y, y_dtype, ldy);
  if (bad != MX_OK || M == 0 || N == 0) return bad;
  const GemvArgs a{x,       ldx, M, w_codes, w_scales, w_scale_ld, nullptr, nullptr, M, N,
                   (int)K,  1,   1, y_dtype == MX_BF16, alpha, y,  ldy,     0,       0};
  return gemv_any<false>(a, x_dtype, M, 1, as_stream(stream));
}

extern "C" int mx_gemv_grouped(const void* x, int x_dtype, int64_t ldx, int64_t x_rows,
                               const int32_t* src, int64_t top_k, const uint8_t* w_codes,
                               const uint8_t* w_scales, int64_t w_scale_ld, const int64_t* offs,
                               int64_t groups, int64_t rows, int64_t N, int64_t K, float alpha,
                               void* y, int y_dtype, int64_t ldy, void* stream) {
  const int bad = gemv_check(x, x_dtype, ldx, w_codes, w_scales, w_scale_ld, rows, N, K, y, y_dtype, ldy);
  if (bad != MX_OK) return bad;
  MX_REQUIRE(groups >= 1 && groups <= MX_MAX_GROUPS && x_rows >= 0 && x_rows <= INT32_MAX &&
                 top_k >= 1 && top_k <= INT32_MAX, MX_ERR_SHAPE);
  if (rows == 0 || N == 0 || x_rows == 0) return MX_OK;
  MX_REQUIRE(offs, MX_ERR_NULL);
  MX_REQUIRE(aligned16(offs) && aligned16(src), MX_ERR_ALIGN);
  const GemvArgs a{x,      ldx,        x_rows,      w_codes, w_scales, w_scale_ld, offs, src, rows, N,
                   (int)K, (int)top_k, (int)groups, y_dtype == MX_BF16, alpha, y, ldy, 0, 0};
  // at most `rows` groups hold rows; their average count picks the row tile
  const int64_t held = hmin(groups, rows);
  return gemv_any<true>(a, x_dtype, cdiv(rows, held), held, as_stream(stream));
}
