// 8-bit quantizers: E4M3 codes with one E8M0 scale per 1x128, 128x1 or 128x128 block, the
// double quantization from rows to columns, and the exact values back.
//
// Rows alone (activations in the forward pass) are read, scaled and written by 16 lanes a block.
// Everything that has columns goes through a 128x128 tile a workgroup: rows and columns come from
// one read (the two operands that a gradient dY gives, the two layouts of a weight).  All of it
// moves bytes and computes little: HBM bandwidth bounds it (a large copy moves 4.8 TB/s, read and
// written).  8192x8192, bf16 and float32: rows 32 and 55 us (6.2 TB/s: two parts in three or four in five
// are reads), columns 32 and 66, both 49 and 82 (5.5 and 4.9), a weight's tiles in both layouts 47 and 80,
// the codes' second quantization 30 (4.5).  Rows that do not start at 16 bytes load twice as much a
// run: 8192x8191 takes 64 and 118 us by rows, 74 and 130 both ways.  Values back from the codes: 31
// and 99 us (6.5 and 3.4 TB/s; one part in three or in five is reads).
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "mx_device8.h"
#include "mx_host8.h"

namespace mx {

// ============================================================== rows
// 16 lanes hold a block, 8 values each; the block's amax is a rotation within the 16 lanes.
// Lanes past the columns hold zeros: they fill the codes up to a multiple of 16 columns, and the
// scale row up to whole dwords.
template <typename T, bool ODD>
__global__ __launch_bounds__(256) void k_quant8_row(const T* __restrict__ x, int64_t ldx, int64_t rows,
                                                    int64_t cols, int per, uint8_t* __restrict__ codes,
                                                    int64_t ld, uint8_t* __restrict__ scales,
                                                    int64_t scale_ld) {
  const int64_t total = rows * per;  // a multiple of 16: whole blocks
  for (int64_t first = (int64_t)blockIdx.x * 256; first < total; first += (int64_t)gridDim.x * 256) {
    if (first + threadIdx.x >= total) continue;
    const RowLane r = row_lane(first, threadIdx.x, per);
    const int64_t col = (int64_t)r.lane * 8;
    Run8<T> run;
    run.template load<ODD>(x + r.row * ldx, col, cols);
    float v[8];
    run.template values<ODD>(col, cols, true, v);
    const uint32_t byte = scale8_byte_of(row16_max_u32(amax_bits<8>(v)));
    if (col - (col & 8) < cols)  // 16 columns with any are written whole
      *reinterpret_cast<uint2*>(codes + r.row * ld + col) = encode8(v, byte);
    const int in = r.lane & 15, block = r.lane >> 4, last = (per >> 4) - 1;
    if (in == 0) scales[r.row * scale_ld + block] = (uint8_t)byte;
    else if (block == last && in <= 3 - (last & 3)) scales[r.row * scale_ld + block + in] = 0;
  }
}

// ============================================================== tiles
// Source of a tile's values: an unquantized matrix, or an 8-bit one by its exact values.
template <typename T, bool ODD>
struct Source8 {
  static constexpr bool kOdd = ODD;
  using Run = Run8<T>;
  const T* x;
  int64_t ld;
  __device__ __forceinline__ void load(Run& r, int64_t row, int64_t col, int64_t cols) const {
    r.template load<ODD>(x + row * ld, col, cols);
  }
  __device__ __forceinline__ void values(const Run& r, int64_t col, int64_t cols, bool there, float v[8]) const {
    r.template values<ODD>(col, cols, there, v);
  }
};
struct CodeRun {
  uint2 codes;
  uint32_t scale;
};
struct Codes8 {  // the codes' columns past cols, up to a multiple of 16, are 0
  using Run = CodeRun;
  const uint8_t* codes;
  const uint8_t* scales;
  int64_t ld, scale_ld;
  __device__ __forceinline__ void load(Run& r, int64_t row, int64_t col, int64_t cols) const {
    const int64_t c = col < cols ? col : 0;
    r.codes = *reinterpret_cast<const uint2*>(codes + row * ld + c);
    r.scale = scales[row * scale_ld + (c >> 7)];
  }
  __device__ __forceinline__ void values(const Run& r, int64_t col, int64_t cols, bool there, float v[8]) const {
    decode8_e4m3(r.codes, scale8_of(r.scale), v);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = there && col + i < cols ? v[i] : 0.0f;
  }
};

// A thread holds 8 rows x 8 columns: rows are loaded and stored 256 (128) bytes wide, a column's 8
// codes of a thread are one 8-byte word of the transposed tile.  That tile goes through LDS, where
// column 8 c + j of a tile lies in row 16 j + c, so that the 16 threads of a row write to
// neighbouring rows, and leaves it in 16-byte pieces, 128 bytes of an output row at a time.
constexpr int kTile8Pitch = 128 + 8;

struct Tile8Lds {
  __align__(16) uint8_t t[128 * kTile8Pitch];
  uint32_t max[4][128];
  uint32_t tile[4];
};

// What a launch makes of a source: its rows' codes and scales, its columns', or both.
template <typename SRC>
struct Tiles8 {
  SRC src;
  int64_t rows, cols;
  uint8_t* codes;
  int64_t ld;
  uint8_t* scales;
  int64_t scale_ld;
  uint8_t* codes_t;
  int64_t ld_t;
  uint8_t* scales_t;
  int64_t scale_ld_t;
};

template <bool TILE, typename SRC>
__device__ __forceinline__ void quant8_tile(const Tiles8<SRC>& q, unsigned block, Tile8Lds& lds) {
  auto& s_t = lds.t;
  auto& s_max = lds.max;
  auto& s_tile = lds.tile;
  const SRC& src = q.src;
  const int64_t rows = q.rows, cols = q.cols, ld = q.ld, scale_ld = q.scale_ld, ld_t = q.ld_t, scale_ld_t = q.scale_ld_t;
  uint8_t *const __restrict__ codes = q.codes, *const __restrict__ scales = q.scales;
  uint8_t *const __restrict__ codes_t = q.codes_t, *const __restrict__ scales_t = q.scales_t;
  const unsigned tiles_c = (unsigned)((cols + 127) / 128);
  const int tid = threadIdx.x, c = tid & 15, rg = tid >> 4, wave = tid >> 6;
  const int64_t tr = block / tiles_c, tc = block % tiles_c;
  const int64_t row0 = tr * 128 + rg * 8, col0 = tc * 128 + c * 8;
  float v[8][8];
  {
    typename SRC::Run run[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) src.load(run[i], row0 + i < rows ? row0 + i : rows - 1, col0, cols);
#pragma unroll
    for (int i = 0; i < 8; ++i) src.values(run[i], col0, cols, row0 + i < rows, v[i]);
  }
  uint32_t tile_byte = 0;
  if constexpr (TILE) {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = max(m, amax_bits<8>(v[i]));
    m = row16_max_u32(m);
    m = max(m, (uint32_t)__shfl_xor((int)m, 16));
    m = max(m, (uint32_t)__shfl_xor((int)m, 32));
    if ((tid & 63) == 0) s_tile[wave] = m;
    __syncthreads();
    tile_byte = scale8_byte_of(max(max(s_tile[0], s_tile[1]), max(s_tile[2], s_tile[3])));
  }
  if (codes) {
    const int64_t blocks = tiles_c;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint32_t byte = TILE ? tile_byte : scale8_byte_of(row16_max_u32(amax_bits<8>(v[i])));
      if (row0 + i < rows) {
        if (col0 - (col0 & 8) < cols)
          *reinterpret_cast<uint2*>(codes + (row0 + i) * ld + col0) = encode8(v[i], byte);
        if (c == 0) scales[(row0 + i) * scale_ld + tc] = (uint8_t)byte;
        else if (tc == blocks - 1 && c <= 3 - ((int)tc & 3)) scales[(row0 + i) * scale_ld + tc + c] = 0;
      }
    }
  }
  if (!codes_t) return;
  uint32_t col_byte[8];
  if constexpr (TILE) {
#pragma unroll
    for (int j = 0; j < 8; ++j) col_byte[j] = tile_byte;
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      float col[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) col[i] = v[i][j];
      uint32_t m = amax_bits<8>(col);
      m = max(m, (uint32_t)__shfl_xor((int)m, 16));
      m = max(m, (uint32_t)__shfl_xor((int)m, 32));
      if ((tid & 48) == 0) s_max[wave][j * 16 + c] = m;
    }
    __syncthreads();
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int at = j * 16 + c;
      col_byte[j] = scale8_byte_of(max(max(s_max[0][at], s_max[1][at]), max(s_max[2][at], s_max[3][at])));
    }
  }
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    float col[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) col[i] = v[i][j];
    *reinterpret_cast<uint2*>(&s_t[(j * 16 + c) * kTile8Pitch + rg * 8]) = encode8(col, col_byte[j]);
  }
  if (rg < 4) {  // thread (rg, c): the scales of columns 8 c + 2 rg and the next, whole dwords at the end
    const int64_t last = (rows + 127) / 128 - 1;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      if ((j >> 1) != rg || col0 + j >= cols) continue;
      uint8_t* p = scales_t + (col0 + j) * scale_ld_t + tr;
      p[0] = (uint8_t)col_byte[j];
      if (tr == last)
        for (int k = 1; k <= 3 - ((int)tr & 3); ++k) p[k] = 0;
    }
  }
  __syncthreads();
  const int64_t rows16 = (rows + 15) / 16 * 16;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const int piece = k * 256 + tid, col = piece >> 3, at = (piece & 7) * 16;
    if (tc * 128 + col >= cols || tr * 128 + at >= rows16) continue;
    const uint8_t* p = &s_t[((col & 7) * 16 + (col >> 3)) * kTile8Pitch + at];
    const uint2 lo = *reinterpret_cast<const uint2*>(p), hi = *reinterpret_cast<const uint2*>(p + 8);
    *reinterpret_cast<uint4*>(codes_t + (tc * 128 + col) * ld_t + tr * 128 + at) =
        make_uint4(lo.x, lo.y, hi.x, hi.y);
  }
}

template <typename SRC, bool TILE>
__global__ __launch_bounds__(256) void k_quant8_tile(const Tiles8<SRC> q) {
  __shared__ Tile8Lds lds;
  quant8_tile<TILE>(q, blockIdx.x, lds);
}

// Two matrices in one launch, the first's tiles in front: what the linear layer quantizes at a time.  A weight
// of 1536x384 has 36 tiles, a twentieth of what the device holds at once (12608 rows, forward and backward,
// 32.6 and 69 us with a launch each, 29.0 and 63 so; 500x384x384 13.7 and 25, 11.4 and 20.5).  At 128 registers
// for a fourth wave a SIMD the float32 tile spills: 8192x8192 both ways 82 us, 116.
template <typename A, bool TILE_A, typename B, bool TILE_B>
__global__ __launch_bounds__(256) void k_quant8_two(const Tiles8<A> a, const Tiles8<B> b, unsigned first) {
  __shared__ Tile8Lds lds;
  if (blockIdx.x < first) quant8_tile<TILE_A>(a, blockIdx.x, lds);
  else quant8_tile<TILE_B>(b, blockIdx.x - first, lds);
}

// ============================================================== values
template <typename T>
__global__ __launch_bounds__(256) void k_dequant8(const Codes8 src, int64_t rows, int64_t cols, int per,
                                                  T* __restrict__ out, int64_t ldo) {
  const int64_t total = rows * per;
  for (int64_t first = (int64_t)blockIdx.x * 256; first < total; first += (int64_t)gridDim.x * 256) {
    if (first + threadIdx.x >= total) continue;
    const RowLane r = row_lane(first, threadIdx.x, per);
    const int64_t col = (int64_t)r.lane * 8;
    CodeRun run;
    src.load(run, r.row, col, cols);
    float v[8];
    src.values(run, col, cols, true, v);
    store8(out + r.row * ldo + col, cols - col, v);
  }
}

// ============================================================== launches
// f(the source of a matrix of this type and number of columns)
template <typename F>
static int with_source8(const void* x, int dtype, int64_t ldx, int64_t cols, F f) {
  const float* p = static_cast<const float*>(x);
  const uint16_t* h = static_cast<const uint16_t*>(x);
  if (dtype == MX_F32) return cols % 8 ? f(Source8<float, true>{p, ldx}) : f(Source8<float, false>{p, ldx});
  return cols % 8 ? f(Source8<uint16_t, true>{h, ldx}) : f(Source8<uint16_t, false>{h, ldx});
}

static unsigned flat_grid(int64_t threads) {
  return (unsigned)hmin(cdiv(threads, 256), (int64_t)device_cu_count() * 64);
}

int quant8_row_impl(const void* x, int dtype, int64_t ldx, int64_t rows, int64_t cols, uint8_t* codes,
                    int64_t ld, uint8_t* scales, int64_t scale_ld, hipStream_t st) {
  if (rows == 0 || cols == 0) return MX_OK;
  const int per = (int)(blocks8(cols) * 16);
  const dim3 grid(flat_grid(rows * per));
#define MX_ROW8(T, ODD)                                                                                        \
  k_quant8_row<T, ODD><<<grid, 256, 0, st>>>(static_cast<const T*>(x), ldx, rows, cols, per, codes, ld, scales, \
                                             scale_ld)
  if (dtype == MX_F32) {
    if (cols % 8) MX_ROW8(float, true);
    else MX_ROW8(float, false);
  } else {
    if (cols % 8) MX_ROW8(uint16_t, true);
    else MX_ROW8(uint16_t, false);
  }
#undef MX_ROW8
  return launch_status();
}

template <typename SRC>
static int64_t tiles8(const Tiles8<SRC>& q) { return blocks8(q.rows) * blocks8(q.cols); }
constexpr int64_t kMaxTiles8 = 0xFFFFFFFFll / 256;  // the work-items of a dispatch

template <bool TILE, typename SRC>
static int launch_tile(const Tiles8<SRC>& q, hipStream_t st) {
  if (q.rows == 0 || q.cols == 0) return MX_OK;
  if (tiles8(q) > kMaxTiles8) return MX_ERR_SHAPE;
  k_quant8_tile<SRC, TILE><<<dim3((unsigned)tiles8(q)), 256, 0, st>>>(q);
  return launch_status();
}

template <bool TILE_A, bool TILE_B, typename A, typename B>
static int launch_two(const Tiles8<A>& a, const Tiles8<B>& b, hipStream_t st) {
  const int64_t first = tiles8(a), blocks = first + tiles8(b);
  if (blocks > kMaxTiles8) return MX_ERR_SHAPE;
  k_quant8_two<A, TILE_A, B, TILE_B><<<dim3((unsigned)blocks), 256, 0, st>>>(a, b, (unsigned)first);
  return launch_status();
}

int quant8_tile_impl(const void* x, int dtype, int64_t ldx, int64_t rows, int64_t cols, bool tile,
                     uint8_t* codes, int64_t ld, uint8_t* scales, int64_t scale_ld, uint8_t* codes_t,
                     int64_t ld_t, uint8_t* scales_t, int64_t scale_ld_t, hipStream_t st) {
  auto run = [&](auto src) {
    const Tiles8<decltype(src)> q{src, rows, cols, codes, ld, scales, scale_ld, codes_t, ld_t, scales_t, scale_ld_t};
    return tile ? launch_tile<true>(q, st) : launch_tile<false>(q, st);
  };
  return with_source8(x, dtype, ldx, cols, run);
}

int requant8_impl(const uint8_t* codes, int64_t ld, const uint8_t* scales, int64_t scale_ld, int64_t rows,
                  int64_t cols, uint8_t* codes_t, int64_t ld_t, uint8_t* scales_t, int64_t scale_ld_t,
                  hipStream_t st) {
  return launch_tile<false>(Tiles8<Codes8>{{codes, scales, ld, scale_ld}, rows, cols, nullptr, 0, nullptr, 0, codes_t,
                                           ld_t, scales_t, scale_ld_t}, st);
}

int quant8_forward_impl(const void* x, int x_dtype, int64_t ldx, int64_t M, const void* w, int w_dtype, int64_t ldw,
                        int64_t N, int64_t K, uint8_t* xq, uint8_t* xs, uint8_t* wq, uint8_t* ws, uint8_t* wt,
                        uint8_t* wts, hipStream_t st) {
  const int64_t ld = round16(K), ls = scale8_pitch(K);
  return with_source8(w, w_dtype, ldw, K, [&](auto sw) {
    return with_source8(x, x_dtype, ldx, K, [&](auto sx) {
      if constexpr (decltype(sw)::kOdd != decltype(sx)::kOdd) return (int)MX_ERR_SHAPE;
      else return launch_two<true, false>(
          Tiles8<decltype(sw)>{sw, N, K, wq, ld, ws, ls, wt, round16(N), wts, scale8_pitch(N)},
          Tiles8<decltype(sx)>{sx, M, K, xq, ld, xs, ls, nullptr, 0, nullptr, 0}, st);
    });
  });
}

int quant8_backward_impl(const void* dy, int dtype, int64_t lddy, int64_t M, int64_t N, const uint8_t* xq,
                         const uint8_t* xs, int64_t K, uint8_t* q, uint8_t* s, uint8_t* qt, uint8_t* qts, uint8_t* xt,
                         uint8_t* xts, hipStream_t st) {
  return with_source8(dy, dtype, lddy, N, [&](auto src) {
    return launch_two<false, false>(
        Tiles8<decltype(src)>{src, M, N, q, round16(N), s, scale8_pitch(N), qt, round16(M), qts, scale8_pitch(M)},
        Tiles8<Codes8>{{xq, xs, round16(K), scale8_pitch(K)}, M, K, nullptr, 0, nullptr, 0, xt, round16(M), xts,
                       scale8_pitch(M)}, st);
  });
}

}  // namespace mx

using namespace mx;

extern "C" int mx_quantize8(const void* x, int dtype, int64_t ldx, int64_t rows, int64_t cols, int axis,
                            uint8_t* codes, int64_t ld, uint8_t* scales, int64_t scale_ld, void* stream) {
  MX_REQUIRE(float_type(dtype) && (axis == MX_ROW || axis == MX_COL), MX_ERR_ENUM);
  MX_REQUIRE(rows >= 0 && cols >= 0 && rows < kMax8 && cols < kMax8 && ldx >= cols, MX_ERR_SHAPE);
  MX_REQUIRE(matrix8(axis == MX_ROW ? cols : rows, ld, scale_ld), MX_ERR_SHAPE);
  if (rows == 0 || cols == 0) return MX_OK;
  MX_REQUIRE(x && codes && scales, MX_ERR_NULL);
  MX_REQUIRE(aligned16(x) && aligned16(codes) && aligned16(scales), MX_ERR_ALIGN);
  if (axis == MX_ROW)
    return quant8_row_impl(x, dtype, ldx, rows, cols, codes, ld, scales, scale_ld, as_stream(stream));
  return quant8_tile_impl(x, dtype, ldx, rows, cols, false, nullptr, 0, nullptr, 0, codes, ld, scales,
                          scale_ld, as_stream(stream));
}

extern "C" int mx_quantize8_dual(const void* x, int dtype, int64_t ldx, int64_t rows, int64_t cols, int tile,
                                 uint8_t* codes, int64_t ld, uint8_t* scales, int64_t scale_ld,
                                 uint8_t* codes_t, int64_t ld_t, uint8_t* scales_t, int64_t scale_ld_t,
                                 void* stream) {
  MX_REQUIRE(float_type(dtype) && (tile == 0 || tile == 1), MX_ERR_ENUM);
  MX_REQUIRE(rows >= 0 && cols >= 0 && rows < kMax8 && cols < kMax8 && ldx >= cols, MX_ERR_SHAPE);
  MX_REQUIRE(matrix8(cols, ld, scale_ld), MX_ERR_SHAPE);
  const bool both = codes_t || scales_t || !tile;  // a weight's second layout may be left out
  if (both) MX_REQUIRE(matrix8(rows, ld_t, scale_ld_t), MX_ERR_SHAPE);
  if (rows == 0 || cols == 0) return MX_OK;
  MX_REQUIRE(x && codes && scales && (!both || (codes_t && scales_t)), MX_ERR_NULL);
  MX_REQUIRE(aligned16(x) && aligned16(codes) && aligned16(scales) && aligned16(codes_t) && aligned16(scales_t),
             MX_ERR_ALIGN);
  return quant8_tile_impl(x, dtype, ldx, rows, cols, tile != 0, codes, ld, scales, scale_ld, codes_t, ld_t,
                          scales_t, scale_ld_t, as_stream(stream));
}

extern "C" int mx_requantize8(const uint8_t* codes, int64_t ld, const uint8_t* scales, int64_t scale_ld,
                              int64_t rows, int64_t cols, uint8_t* codes_t, int64_t ld_t, uint8_t* scales_t,
                              int64_t scale_ld_t, void* stream) {
  MX_REQUIRE(rows >= 0 && cols >= 0 && rows < kMax8 && cols < kMax8, MX_ERR_SHAPE);
  if (rows == 0 || cols == 0) return MX_OK;
  MX_REQUIRE(matrix8(cols, ld, scale_ld) && matrix8(rows, ld_t, scale_ld_t), MX_ERR_SHAPE);
  MX_REQUIRE(codes && scales && codes_t && scales_t, MX_ERR_NULL);
  MX_REQUIRE(aligned16(codes) && aligned16(scales) && aligned16(codes_t) && aligned16(scales_t), MX_ERR_ALIGN);
  return requant8_impl(codes, ld, scales, scale_ld, rows, cols, codes_t, ld_t, scales_t, scale_ld_t,
                       as_stream(stream));
}

extern "C" int mx_dequantize8(const uint8_t* codes, int64_t ld, const uint8_t* scales, int64_t scale_ld,
                              int64_t rows, int64_t cols, void* out, int out_dtype, int64_t ldo, void* stream) {
  MX_REQUIRE(float_type(out_dtype), MX_ERR_ENUM);
  MX_REQUIRE(rows >= 0 && cols >= 0 && rows < kMax8 && cols < kMax8 && ldo >= cols, MX_ERR_SHAPE);
  if (rows == 0 || cols == 0) return MX_OK;
  MX_REQUIRE(matrix8(cols, ld, scale_ld), MX_ERR_SHAPE);
  MX_REQUIRE(codes && scales && out, MX_ERR_NULL);
  MX_REQUIRE(aligned16(codes) && aligned16(scales) && aligned16(out), MX_ERR_ALIGN);
  const int per = (int)cdiv(cols, 8);
  const dim3 grid(flat_grid(rows * per));
  const Codes8 src{codes, scales, ld, scale_ld};
  if (out_dtype == MX_F32)
    k_dequant8<float><<<grid, 256, 0, as_stream(stream)>>>(src, rows, cols, per, static_cast<float*>(out), ldo);
  else
    k_dequant8<uint16_t><<<grid, 256, 0, as_stream(stream)>>>(src, rows, cols, per, static_cast<uint16_t*>(out),
                                                              ldo);
  return launch_status();
}
