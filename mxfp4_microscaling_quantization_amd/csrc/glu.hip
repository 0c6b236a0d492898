// Gated activation between the up and the down product of a (mixture-of-experts) MLP, and its
// gradient from an 8-bit checkpoint:
//   z = (g, u), h = act(g) u;   dg = dh u act'(g), du = dh act(g)
// with g and u of the backward pass as the checkpoint holds them.  act is g / (1 + e^-g) or
// g Phi(g), Phi the normal distribution.
//
// One read of z gives h -- in float32, bf16, or already as the packed 4-bit or 8-bit operand of
// the next product -- and the checkpoint: the 8-bit matrix of the rows' halves, 2 1/64 bytes a
// column of h instead of the 4 or 8 of z.  16 lanes hold 128 columns of a half, 8 values a lane,
// so the blocks' maxima are rotations within the 16.  All of it is bound by HBM: 65536x2880, float32 z, as MXFP4
// operand 320 us (5.0 TB/s), with the checkpoint 399; bf16 z 205 (4.2) and 274, GELU 224 and 294.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "mx_device8.h"
#include "mx_host8.h"

namespace mx {

// Rows of a buffer that are in use: all, or as many as a device counter says.
__device__ __forceinline__ int64_t live_rows(const int64_t* __restrict__ live, int64_t rows) {
  if (!live) return rows;
  const int64_t n = *live;
  return n < 0 ? 0 : (n < rows ? n : rows);
}

// Phi(g), and e^(-g^2/2).  With a = |g|, Phi(-a) = e^(-a^2/2) t Q(t), t = 1 / (1 + 0.35 a): Q is the polynomial of
// degree 8 with the smallest relative error at the Chebyshev points of a <= 15 (weighted least squares with
// Lawson's weights), 3.2e-8, and with these rounded coefficients 7 * 2^-24 in Phi.  a^2 is carried to its
// last bit into the exponential.  Beyond a of 15 both are 0.  The library's erfcf with an exponential of its own took
// 397 us for the gradient of 65536x2880 where SILU takes 283; 302 so.
__device__ __forceinline__ float normal_below(float g, float* e) {
  const float a = fminf(fabsf(g), 30.0f), t = __builtin_amdgcn_rcpf(fmaf(a, 0.35f, 1.0f));
  float q = -0.0291638058f;
  q = fmaf(q, t, 0.144060239f);
  q = fmaf(q, t, -0.255900741f);
  q = fmaf(q, t, 0.159391701f);
  q = fmaf(q, t, -0.0232630335f);
  q = fmaf(q, t, 0.105574481f);
  q = fmaf(q, t, 0.119815573f);
  q = fmaf(q, t, 0.139864326f);
  q = fmaf(q, t, 0.139621258f);
  const float square = a * a, rest = fmaf(a, a, -square);
  *e = expf(-0.5f * square);
  *e = fmaf(*e, -0.5f * rest, *e);
  const float below = q * t * *e;
  return g < 0.0f ? below : 1.0f - below;
}

// act(g); with D also its derivative.
template <bool D>
__device__ __forceinline__ float activate(float g, int act, float* d) {
  if (act == MX_SILU) {
    const float s = 1.0f / (1.0f + expf(-g));
    if (D) *d = s + s * (g * (1.0f - s));
    return g * s;
  }
  float e;
  const float phi = normal_below(g, &e);
  if (D) *d = phi + g * (0.39894228040143268f * e);
  return g * phi;
}

struct Packed8 {  // an 8-bit matrix to write or to read
  uint8_t* codes;
  uint8_t* scales;
  int64_t ld, scale_ld;
  // a lane's 8 columns of row `row`, the block's byte, and the row's last bytes
  __device__ __forceinline__ void store(int64_t row, int lane, int64_t cols, int per, const float v[8]) const {
    const uint32_t byte = scale8_byte_of(row16_max_u32(amax_bits<8>(v)));
    const int64_t col = (int64_t)lane * 8;
    if (col - (col & 8) < cols) *reinterpret_cast<uint2*>(codes + row * ld + col) = encode8(v, byte);
    const int in = lane & 15, block = lane >> 4, last = (per >> 4) - 1;
    if (in == 0) scales[row * scale_ld + block] = (uint8_t)byte;
    else if (block == last && in <= 3 - (last & 3)) scales[row * scale_ld + block + in] = 0;
  }
};

// What becomes of h: values, or an operand of the next product.
template <typename T>
struct OutValues {
  T* p;
  int64_t ld;
  __device__ __forceinline__ void store(int64_t row, int lane, int64_t cols, int, const float v[8]) const {
    const int64_t col = (int64_t)lane * 8;
    store8(p + row * ld + col, cols - col, v);
  }
};
struct OutPacked4 {  // Q_D with 1x32 blocks, a quad of lanes a block; cols % 32 == 0
  uint32_t* codes;
  uint8_t* scales;
  int64_t scale_ld;
  __device__ __forceinline__ void store(int64_t row, int lane, int64_t cols, int, const float v[8]) const {
    const uint32_t byte = scale_byte_of(quad_max_u32(amax_bits<8>(v)));
    if (lane * 8 >= cols) return;
    uint32_t w = 0;
    if (byte != 255u) {
      const float sc = scale_of(byte);
#pragma unroll
      for (int i = 0; i < 4; ++i) w |= (cvt_rne_pair(v[2 * i], v[2 * i + 1], sc) & 0xFFu) << (8 * i);
    }
    codes[row * (cols / 8) + lane] = w;
    if ((lane & 3) == 0) scales[row * scale_ld + (lane >> 2)] = (uint8_t)byte;
  }
};

template <typename T, typename OUT, bool KEEP, bool ODD>
__global__ __launch_bounds__(256) void k_glu(const T* __restrict__ z, int64_t ldz,
                                             const int64_t* __restrict__ live, int64_t rows, int64_t cols,
                                             int per, int act, const OUT out, const Packed8 kept) {
  const int64_t total = live_rows(live, rows) * per;  // a multiple of 16: whole blocks
  for (int64_t first = (int64_t)blockIdx.x * 256; first < total; first += (int64_t)gridDim.x * 256) {
    if (first + threadIdx.x >= total) continue;
    const RowLane r = row_lane(first, threadIdx.x, per);
    const int64_t col = (int64_t)r.lane * 8;
    const T* p = z + r.row * ldz;
    Run8<T> gate, up;
    gate.template load<ODD>(p, col, cols);
    up.template load<ODD>(p + cols, col, cols);
    float g[8], u[8], h[8];
    gate.template values<ODD>(col, cols, true, g);
    up.template values<ODD>(col, cols, true, u);
#pragma unroll
    for (int i = 0; i < 8; ++i) h[i] = activate<false>(g[i], act, nullptr) * u[i];
    out.store(r.row, r.lane, cols, per, h);
    if constexpr (KEEP) {
      kept.store(2 * r.row, r.lane, cols, per, g);
      kept.store(2 * r.row + 1, r.lane, cols, per, u);
    }
  }
}

template <typename TH, typename TZ, bool ODD>
__global__ __launch_bounds__(256) void k_glu_bwd(const TH* __restrict__ dh, int64_t lddh, const Packed8 kept,
                                                 const int64_t* __restrict__ live, int64_t rows, int64_t cols,
                                                 int per, int act, TZ* __restrict__ dz, int64_t lddz) {
  const int64_t total = live_rows(live, rows) * per;
  for (int64_t first = (int64_t)blockIdx.x * 256; first < total; first += (int64_t)gridDim.x * 256) {
    if (first + threadIdx.x >= total) continue;
    const RowLane r = row_lane(first, threadIdx.x, per);
    const int64_t col = (int64_t)r.lane * 8, n = cols - col;
    const uint8_t* c = kept.codes + 2 * r.row * kept.ld + col;
    const uint8_t* s = kept.scales + 2 * r.row * kept.scale_ld + (col >> 7);
    const uint2 gate = *reinterpret_cast<const uint2*>(c), up = *reinterpret_cast<const uint2*>(c + kept.ld);
    const uint32_t gate_scale = s[0], up_scale = s[kept.scale_ld];
    Run8<TH> run;
    run.template load<ODD>(dh + r.row * lddh, col, cols);
    float g[8], u[8], d[8];
    decode8_e4m3(gate, scale8_of(gate_scale), g);
    decode8_e4m3(up, scale8_of(up_scale), u);
    run.template values<ODD>(col, cols, true, d);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      float da;
      const float a = activate<true>(g[i], act, &da);
      g[i] = d[i] * u[i] * da;
      u[i] = d[i] * a;
    }
    TZ* p = dz + r.row * lddz + col;
    store8(p, n, g);
    store8(p + cols, n, u);
  }
}

// ============================================================== launches
static unsigned glu_grid(int64_t threads) {
  return (unsigned)hmin(cdiv(threads, 256), (int64_t)device_cu_count() * 64);
}

template <typename OUT>
static int launch_glu(const void* z, int z_dtype, int64_t ldz, const int64_t* live, int64_t rows, int64_t cols,
                      int act, const OUT& out, const Packed8& kept, hipStream_t st) {
  const int per = (int)(blocks8(cols) * 16);
  const dim3 grid(glu_grid(rows * per));
#define MX_GLU_ODD(T, KEEP, ODD) \
  k_glu<T, OUT, KEEP, ODD><<<grid, 256, 0, st>>>(static_cast<const T*>(z), ldz, live, rows, cols, per, act, out, kept)
#define MX_GLU(T, KEEP)                     \
  do {                                      \
    if (cols % 8) MX_GLU_ODD(T, KEEP, true); \
    else MX_GLU_ODD(T, KEEP, false);         \
  } while (0)
  if (z_dtype == MX_F32) {
    if (kept.codes) MX_GLU(float, true);
    else MX_GLU(float, false);
  } else {
    if (kept.codes) MX_GLU(uint16_t, true);
    else MX_GLU(uint16_t, false);
  }
#undef MX_GLU
#undef MX_GLU_ODD
  return launch_status();
}

static bool glu_shape(int64_t rows, int64_t cols) {
  return rows >= 0 && rows < kMax8 / 2 && cols >= 0 && cols <= kMaxAxis8;
}

// What the three forward calls share; MX_OK with nothing to do is told by rows or cols of 0.
static int check_glu(const void* z, int z_dtype, int64_t ldz, const int64_t* live, int64_t rows, int64_t cols,
                     int act, const Packed8& kept) {
  MX_REQUIRE(float_type(z_dtype) && (act == MX_SILU || act == MX_GELU), MX_ERR_ENUM);
  MX_REQUIRE(glu_shape(rows, cols) && ldz >= 2 * cols, MX_ERR_SHAPE);
  const bool keep = kept.codes || kept.scales;
  if (keep) MX_REQUIRE(matrix8(cols, kept.ld, kept.scale_ld), MX_ERR_SHAPE);
  if (rows == 0 || cols == 0) return MX_OK;
  MX_REQUIRE(z && (!keep || (kept.codes && kept.scales)), MX_ERR_NULL);
  MX_REQUIRE(aligned16(z) && aligned16(kept.codes) && aligned16(kept.scales) &&
                 (reinterpret_cast<uintptr_t>(live) & 7) == 0, MX_ERR_ALIGN);
  return MX_OK;
}

}  // namespace mx

using namespace mx;

extern "C" int mx_glu(const void* z, int z_dtype, int64_t ldz, const int64_t* live, int64_t rows, int64_t cols,
                      int act, void* h, int h_dtype, int64_t ldh, uint8_t* kept_codes, int64_t kept_ld,
                      uint8_t* kept_scales, int64_t kept_scale_ld, void* stream) {
  const Packed8 kept{kept_codes, kept_scales, kept_ld, kept_scale_ld};
  MX_REQUIRE(float_type(h_dtype), MX_ERR_ENUM);
  const int s = check_glu(z, z_dtype, ldz, live, rows, cols, act, kept);
  if (s != MX_OK) return s;
  MX_REQUIRE(ldh >= cols, MX_ERR_SHAPE);
  if (rows == 0 || cols == 0) return MX_OK;
  MX_REQUIRE(h, MX_ERR_NULL);
  MX_REQUIRE(aligned16(h), MX_ERR_ALIGN);
  if (h_dtype == MX_F32)
    return launch_glu(z, z_dtype, ldz, live, rows, cols, act, OutValues<float>{static_cast<float*>(h), ldh}, kept,
                      as_stream(stream));
  return launch_glu(z, z_dtype, ldz, live, rows, cols, act, OutValues<uint16_t>{static_cast<uint16_t*>(h), ldh},
                    kept, as_stream(stream));
}

extern "C" int mx_glu_quantize(const void* z, int z_dtype, int64_t ldz, const int64_t* live, int64_t rows,
                               int64_t cols, int act, uint8_t* codes, uint8_t* scales, int64_t scale_ld,
                               uint8_t* kept_codes, int64_t kept_ld, uint8_t* kept_scales,
                               int64_t kept_scale_ld, void* stream) {
  const Packed8 kept{kept_codes, kept_scales, kept_ld, kept_scale_ld};
  const int s = check_glu(z, z_dtype, ldz, live, rows, cols, act, kept);
  if (s != MX_OK) return s;
  MX_REQUIRE(cols % 32 == 0 && scale_ld >= cols / 32, MX_ERR_SHAPE);
  if (rows == 0 || cols == 0) return MX_OK;
  MX_REQUIRE(codes && scales, MX_ERR_NULL);
  MX_REQUIRE(aligned16(codes) && aligned16(scales), MX_ERR_ALIGN);
  return launch_glu(z, z_dtype, ldz, live, rows, cols, act,
                    OutPacked4{reinterpret_cast<uint32_t*>(codes), scales, scale_ld}, kept, as_stream(stream));
}

extern "C" int mx_glu_quantize8(const void* z, int z_dtype, int64_t ldz, const int64_t* live, int64_t rows,
                                int64_t cols, int act, uint8_t* codes, int64_t ld, uint8_t* scales,
                                int64_t scale_ld, uint8_t* kept_codes, int64_t kept_ld, uint8_t* kept_scales,
                                int64_t kept_scale_ld, void* stream) {
  const Packed8 kept{kept_codes, kept_scales, kept_ld, kept_scale_ld};
  const int s = check_glu(z, z_dtype, ldz, live, rows, cols, act, kept);
  if (s != MX_OK) return s;
  MX_REQUIRE(matrix8(cols, ld, scale_ld), MX_ERR_SHAPE);
  if (rows == 0 || cols == 0) return MX_OK;
  MX_REQUIRE(codes && scales, MX_ERR_NULL);
  MX_REQUIRE(aligned16(codes) && aligned16(scales), MX_ERR_ALIGN);
  return launch_glu(z, z_dtype, ldz, live, rows, cols, act, Packed8{codes, scales, ld, scale_ld}, kept,
                    as_stream(stream));
}

extern "C" int mx_glu_bwd(const void* dh, int dh_dtype, int64_t lddh, const uint8_t* kept_codes, int64_t kept_ld,
                          const uint8_t* kept_scales, int64_t kept_scale_ld, const int64_t* live, int64_t rows,
                          int64_t cols, int act, void* dz, int dz_dtype, int64_t lddz, void* stream) {
  MX_REQUIRE(float_type(dh_dtype) && float_type(dz_dtype) && (act == MX_SILU || act == MX_GELU), MX_ERR_ENUM);
  MX_REQUIRE(glu_shape(rows, cols) && lddh >= cols && lddz >= 2 * cols && matrix8(cols, kept_ld, kept_scale_ld),
             MX_ERR_SHAPE);
  if (rows == 0 || cols == 0) return MX_OK;
  MX_REQUIRE(dh && kept_codes && kept_scales && dz, MX_ERR_NULL);
  MX_REQUIRE(aligned16(dh) && aligned16(kept_codes) && aligned16(kept_scales) && aligned16(dz) &&
                 (reinterpret_cast<uintptr_t>(live) & 7) == 0, MX_ERR_ALIGN);
  const int per = (int)cdiv(cols, 8);
  const dim3 grid(glu_grid(rows * per));
  const hipStream_t st = as_stream(stream);
  const Packed8 kept{const_cast<uint8_t*>(kept_codes), const_cast<uint8_t*>(kept_scales), kept_ld, kept_scale_ld};
#define MX_GLU_BWD_ODD(TH, TZ, ODD)                                                                          \
  k_glu_bwd<TH, TZ, ODD><<<grid, 256, 0, st>>>(static_cast<const TH*>(dh), lddh, kept, live, rows, cols, per, act, \
                                               static_cast<TZ*>(dz), lddz)
#define MX_GLU_BWD(TH, TZ)                     \
  do {                                         \
    if (cols % 8) MX_GLU_BWD_ODD(TH, TZ, true); \
    else MX_GLU_BWD_ODD(TH, TZ, false);         \
  } while (0)
  if (dh_dtype == MX_F32) {
    if (dz_dtype == MX_F32) MX_GLU_BWD(float, float);
    else MX_GLU_BWD(float, uint16_t);
  } else {
    if (dz_dtype == MX_F32) MX_GLU_BWD(uint16_t, float);
    else MX_GLU_BWD(uint16_t, uint16_t);
  }
#undef MX_GLU_BWD
#undef MX_GLU_BWD_ODD
  return launch_status();
}
