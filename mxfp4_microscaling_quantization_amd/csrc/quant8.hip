// 8-bit quantizers: E4M3 codes with one E8M0 scale per 1x128, 128x1 or 128x128 block, the
// double quantization from rows to columns, and the exact values back.
//
// Rows alone (activations in the forward pass) are read, scaled and written by 16 lanes a block.
// Everything that has columns goes through a 128x128 tile a workgroup: rows and columns come from
// one read (the two operands that a gradient dY gives, the two layouts of a weight).  All of it
// moves bytes and computes little: HBM bandwidth bounds it.
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

template <typename SRC, bool TILE>
__global__ __launch_bounds__(256) void k_quant8_tile(const SRC src, int64_t rows, int64_t cols,
                                                     int64_t tiles_c, uint8_t* __restrict__ codes,
                                                     int64_t ld, uint8_t* __restrict__ scales,
                                                     int64_t scale_ld, uint8_t* __restrict__ codes_t,
                                                     int64_t ld_t, uint8_t* __restrict__ scales_t,
                                                     int64_t scale_ld_t) {
  __shared__ __align__(16) uint8_t s_t[128 * kTile8Pitch];
  __shared__ uint32_t s_max[4][128];
  __shared__ uint32_t s_tile[4];
  const int tid = threadIdx.x, c = tid & 15, rg = tid >> 4, wave = tid >> 6;
  const int64_t tr = blockIdx.x / tiles_c, tc = blockIdx.x % tiles_c;
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

template <bool TILE, typename SRC>
static int launch_tile(const SRC& src, int64_t rows, int64_t cols, uint8_t* codes, int64_t ld, uint8_t* scales,
                       int64_t scale_ld, uint8_t* codes_t, int64_t ld_t, uint8_t* scales_t, int64_t scale_ld_t,
                       hipStream_t st) {
  if (rows == 0 || cols == 0) return MX_OK;
  const int64_t tiles_c = blocks8(cols), tiles = blocks8(rows) * tiles_c;
  if (tiles > 0xFFFFFFFFll / 256) return MX_ERR_SHAPE;  // the work-items of a dispatch
  k_quant8_tile<SRC, TILE><<<dim3((unsigned)tiles), 256, 0, st>>>(src, rows, cols, tiles_c, codes, ld, scales,
                                                                  scale_ld, codes_t, ld_t, scales_t, scale_ld_t);
  return launch_status();
}

int quant8_tile_impl(const void* x, int dtype, int64_t ldx, int64_t rows, int64_t cols, bool tile,
                     uint8_t* codes, int64_t ld, uint8_t* scales, int64_t scale_ld, uint8_t* codes_t,
                     int64_t ld_t, uint8_t* scales_t, int64_t scale_ld_t, hipStream_t st) {
#define MX_TILE8_ODD(T, TILE, ODD)                                                                        \
  launch_tile<TILE>(Source8<T, ODD>{static_cast<const T*>(x), ldx}, rows, cols, codes, ld, scales, scale_ld, \
                    codes_t, ld_t, scales_t, scale_ld_t, st)
#define MX_TILE8(T, TILE) (cols % 8 ? MX_TILE8_ODD(T, TILE, true) : MX_TILE8_ODD(T, TILE, false))
  if (dtype == MX_F32) return tile ? MX_TILE8(float, true) : MX_TILE8(float, false);
  return tile ? MX_TILE8(uint16_t, true) : MX_TILE8(uint16_t, false);
#undef MX_TILE8
#undef MX_TILE8_ODD
}

int requant8_impl(const uint8_t* codes, int64_t ld, const uint8_t* scales, int64_t scale_ld, int64_t rows,
                  int64_t cols, uint8_t* codes_t, int64_t ld_t, uint8_t* scales_t, int64_t scale_ld_t,
                  hipStream_t st) {
  return launch_tile<false>(Codes8{codes, scales, ld, scale_ld}, rows, cols, nullptr, 0, nullptr, 0, codes_t,
                            ld_t, scales_t, scale_ld_t, st);
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
